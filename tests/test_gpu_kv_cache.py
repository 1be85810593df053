"""The paged key/value cache and its attention on a GB300, against their definitions in 64 bits
(tests/kv_util.py, which derives the tolerances)."""
import math

import pytest
import torch

import tests.kv_util as U
from mixture_experts_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 128), ("bf16", 256), ("bf16", 512), ("e4m3", 128), ("e4m3", 256), ("e4m3", 512)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def _ok(kv):
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_OK, 0)


# ------------------------------------------------------------------ writing and reading back

def _expected_cache(case, kv, c):
    """The cache's tensors after case.filled, in the same order: values, and scales."""
    want = case.empty_cache(kv)
    for b, n in enumerate(case.kv):
        for p in range(n):
            page, slot = int(case.pages[b, p // case.page]), p % case.page
            for name, x in (("k", case.k[b][p]), ("v", case.v[b][p])):
                t = getattr(want, name)
                if case.fmt == "bf16":
                    t[page, :, slot] = x.cuda()
                else:
                    codes, scale = U.quantised(x)
                    t.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8).cuda()
                    getattr(want, name + "_scale")[page, :, slot] = scale.cuda()
    return want


def _same_bits(a, b):
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    a, b = a.view(kind), b.view(kind)
    assert torch.equal(a, b), "%d of %d values differ" % ((a != b).sum(), a.numel())


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("page,hkv", [(16, 1), (32, 3), (64, 8), (128, 2)])
def test_written_bits(fmt, d, page, hkv):
    case = U.Case(fmt, hkv, hkv, d, page, [0] * 4, [1, page, page + 1, 2 * page + 5], seed=d + page, garbage="zero")
    case.k[3][7] = 0.0                       # a row of zeros
    case.k[3][8] *= 2.0 ** -120              # near the bottom of bf16's range
    case.v[3][9] *= 2.0 ** 120
    kv = case.handle()
    c = case.filled(kv)
    _ok(kv)
    want = _expected_cache(case, kv, c)
    for n in ("k", "v") + (("k_scale", "v_scale") if fmt == "e4m3" else ()):
        _same_bits(getattr(c, n), getattr(want, n))


@pytest.mark.parametrize("fmt,d", SHAPES)
def test_round_trip(fmt, d):
    case = U.Case(fmt, 4, 2, d, 16, [3, 0, 17, 1], [3, 40, 30, 100], seed=d, pad_rows=2)
    kv = case.handle()
    c = case.filled(kv)
    k, v = kv.read(c, case.batch(), n_tokens=case.T)
    _ok(kv)
    for name, got in (("k", k), ("v", v)):
        want = torch.cat([case.stored(name, b)[case.kv[b] - n:] for b, n in enumerate(case.new)]
                         + [torch.zeros(2, case.hkv, d, dtype=torch.float64)])
        U.check_close(got, want, (U.BF + U.F32) * want.abs() if fmt == "e4m3" else torch.zeros_like(want), name)
    assert torch.equal(kv.read(c, case.batch())[0], k[:case.cu[-1]])


def test_rows_with_infinities_read_back_as_nan_in_e4m3():
    case = U.Case("e4m3", 2, 2, 256, 32, [0], [9], seed=1)
    case.k[0][3, 1, 17] = math.inf
    case.v[0][5, 0, 255] = math.nan
    kv = case.handle()
    c = case.filled(kv)
    k, v = kv.read(c, case.batch([9]), n_tokens=9)
    _ok(kv)
    for got, at in ((k, (3, 1)), (v, (5, 0))):
        nan = torch.isnan(got).all(-1)
        assert nan[at] and nan.sum() == 1 and torch.isnan(got).any(-1).sum() == 1


def test_strided_views_write_the_same():
    case = U.Case("e4m3", 4, 4, 256, 32, [0, 0], [37, 20], seed=2)
    kv = case.handle()
    base = case.filled(kv)
    k, v = torch.cat(case.k).cuda(), torch.cat(case.v).cuda()
    T = k.shape[0]
    fused = torch.zeros(T, 3, 4, 256, dtype=torch.bfloat16, device="cuda")
    fused[:, 1], fused[:, 2] = k, v
    other = case.empty_cache(kv)
    kv.write(other, case.batch([37, 20]), fused[:, 1], v.transpose(0, 1).contiguous().transpose(0, 1))
    _ok(kv)
    for n in ("k", "v", "k_scale", "v_scale"):
        _same_bits(getattr(base, n), getattr(other, n))


def test_tokens_of_no_position_write_nothing():
    # Three new tokens of a sequence whose cache holds two, and padding rows.
    case = U.Case("bf16", 2, 2, 128, 16, [3, 1], [2, 1], seed=3, pad_rows=3, garbage="zero")
    kv = case.handle()
    c = kv.new_cache()
    x = torch.randn(7, 2, 128, device="cuda").to(torch.bfloat16)
    kv.write(c, case.batch(), x, -x)
    _ok(kv)
    assert (c.k != 0).any(-1).sum() == 3 * 2
    page = int(case.pages[0, 0])
    assert torch.equal(c.k[page, :, :2].transpose(0, 1), x[1:3])
    k, _ = kv.read(c, case.batch(), n_tokens=7)
    assert torch.equal(k[1:4], x[1:4]) and not k[0].any() and not k[4:].any()


@pytest.mark.parametrize("n_seqs", [1, 31, 33, 300, 1100])
def test_many_sequences_find_their_places(n_seqs):
    new = [(7 * b) % 3 for b in range(n_seqs)]
    case = U.Case("bf16", 1, 1, 128, 16, new, [n + (5 * b) % 40 for b, n in enumerate(new)], seed=4, pad_rows=1)
    kv = case.handle()
    c = case.filled(kv)
    k, v = kv.read(c, case.batch(), n_tokens=case.T)
    _ok(kv)
    for got, have in ((k, case.k), (v, case.v)):
        want = torch.cat([have[b][case.kv[b] - n:] for b, n in enumerate(new)] + [torch.zeros(1, 1, 128).bfloat16()])
        assert torch.equal(got.cpu(), want)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("page", [16, 128])
def test_single_tokens(fmt, d, page):
    kv_len = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]
    U.check_attention(U.Case(fmt, 4, 2, d, page, [1] * len(kv_len), kv_len, seed=d))


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("group", [1, 3, 8, 11])
def test_head_groups(fmt, d, group):
    U.check_attention(U.Case(fmt, 2 * group, 2, d, 32, [1, 1, 1], [40, 1, 150], seed=group))
    U.check_attention(U.Case(fmt, 2 * group, 2, d, 32, [5, 1, 30], [40, 1, 130], seed=group))


@pytest.mark.parametrize("fmt,d", SHAPES)
def test_chunks(fmt, d):
    U.check_attention(U.Case(fmt, 4, 2, d, 16, [1, 64, 65, 7, 0, 130], [1, 64, 200, 263, 90, 131], seed=d))


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (20, 0), (64, 4), (100, 40), (100, 1000), (1000, 4)])
def test_windows_and_sinks(fmt, d, window, sinks):
    U.check_attention(U.Case(fmt, 2, 1, d, 16, [1, 1, 1, 1], [1, 20, 21, 333], seed=window), window, sinks)
    U.check_attention(U.Case(fmt, 2, 1, d, 16, [130, 3, 77], [130, 300, 211], seed=window), window, sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [0, 5, 0]), ([4, 1, 70], [2, 0, 33]), ([0, 0], [7, 0])])
def test_rows_that_see_nothing(fmt, new, kv):
    case = U.Case(fmt, 4, 2, 256, 16, new, kv, seed=5, pad_rows=3)
    out, lse = U.check_attention(case, window=9)
    assert not out[case.cu[-1]:].any() and torch.isinf(lse[case.cu[-1]:]).all()


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
def test_hidden_values_do_not_matter(fmt, d, window, sinks):
    """NaN and infinities in keys and values change only the rows that see them."""
    case = U.Case(fmt, 2, 1, d, 16, [90, 1], [150, 200], seed=6)
    case.v[0][130, 0, 5] = math.nan
    case.v[0][100, 0, d - 1] = math.inf
    case.k[0][145, 0, 3] = math.nan
    case.v[0][30, 0, 40] = math.nan       # outside every window but the first rows'
    case.k[1][20, 0, 3] = math.nan        # hidden by the window
    U.check_attention(case, window, sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_queries_with_nan_stay_alone(fmt):
    case = U.Case(fmt, 4, 2, 256, 32, [20, 1], [50, 77], seed=7)
    case.q[3, 1, 0] = math.nan
    case.q[20, 2, 9] = math.nan
    U.check_attention(case)


@pytest.mark.parametrize("fmt,d", [("bf16", 256), ("e4m3", 512)])
def test_large_scores(fmt, d):
    # Scores of some hundreds: the running maximum moves far and often.
    case = U.Case(fmt, 2, 1, d, 16, [60, 1], [200, 500], seed=8)
    for k in case.k:
        k.mul_(torch.linspace(0.2, 8, k.shape[0]).view(-1, 1, 1))
    case.q.mul_(6)
    U.check_attention(case)


def test_scale_and_strided_queries():
    case = U.Case("bf16", 6, 2, 128, 32, [9, 1], [40, 60], seed=9)
    fused = torch.zeros(10, 10, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 2:8] = case.q.cuda()
    U.check_attention(case, scale=0.3, q=fused[:, 2:8])
    by_head = case.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    U.check_attention(case, scale=0.01, q=by_head)


def _large(fmt, hq, hkv, d, page, new, kv, seed):
    """A case too large for the row-by-row definition, and its result by 64-bit products on the GPU."""
    case = U.Case(fmt, hq, hkv, d, page, new, kv, seed=seed)
    h = case.handle()
    c = case.filled(h)
    g = hq // hkv

    def want(window, sinks):
        out, lse = [], []
        for b, n in enumerate(new):
            k, v = case.stored("k", b).cuda(), case.stored("v", b).cuda()
            q = case.q[case.cu[b]:case.cu[b + 1]].double().cuda()
            s = torch.einsum("thd,jhd->htj", q, k.repeat_interleave(g, 1)) * d ** -0.5
            j, p = torch.arange(kv[b], device="cuda"), torch.arange(kv[b] - n, kv[b], device="cuda")[:, None]
            see = j <= p
            if window:
                see = see & ((j > p - window) | (j < sinks))
            s = s.masked_fill(~see, -math.inf)
            out.append(torch.einsum("htj,jhd->thd", torch.softmax(s, -1), v.repeat_interleave(g, 1)))
            lse.append(torch.logsumexp(s, -1).T)
        return torch.cat(out).cpu(), torch.cat(lse).cpu()

    return case, h, c, want


@pytest.mark.parametrize("fmt,hq,hkv,d,page,new,kv", [
    ("bf16", 16, 2, 512, 64, [1, 1], [20011, 3]), ("e4m3", 16, 8, 256, 16, [1] * 5, [5000, 1, 900, 2048, 4097]),
    ("bf16", 8, 2, 128, 128, [40, 3], [9000, 30]), ("e4m3", 4, 1, 512, 32, [300], [5000]),
    ("bf16", 16, 8, 256, 64, [700, 1, 129], [2000, 1999, 129])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1024, 4)])
def test_long_caches(fmt, hq, hkv, d, page, new, kv, window, sinks):
    case, h, c, want = _large(fmt, hq, hkv, d, page, new, kv, seed=10)
    out, lse = h.attention(c, case.batch(), case.q.cuda(), window=window, sinks=sinks)
    _ok(h)
    w, wl = want(window, sinks)
    # Values of order 1 under softmax weights that sum to 1: one rounding of the weights, 2^-8 of what
    # they weigh, and one of the result; 2^-10 for everything held in fp32.
    U.check_close(lse, wl, torch.full_like(wl, 2.0 ** -10), "lse")
    U.check_close(out, w, 2 * U.BF * w.abs() + U.BF + 2.0 ** -10, "out")
    out2, lse2 = h.attention(c, case.batch(), case.q.cuda(), window=window, sinks=sinks)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
def test_hidden_values_do_not_matter_to_single_tokens(fmt, d, window, sinks):
    case = U.Case(fmt, 3, 1, d, 16, [1, 1, 1], [150, 200, 33], seed=16)
    case.v[0][149, 0, 5] = math.nan        # seen
    case.v[0][100, 0, d - 1] = math.nan    # hidden by the window
    case.k[1][50, 0, 3] = math.nan
    case.v[1][1, 0, 7] = math.inf          # a sink
    U.check_attention(case, window, sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_hidden_values_with_one_head_per_kv_head(fmt):
    """Row tiles of 256 tokens: keys that some rows see lie up to 255 from the first."""
    case = U.Case(fmt, 1, 1, 128, 32, [300], [420], seed=17)
    for p in (121, 250, 374, 375, 376, 419):
        case.v[0][p, 0, p % 128] = math.nan
    U.check_attention(case)
    U.check_attention(case, 130, 3)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n_seqs", [300, 1300])
def test_many_sequences(fmt, n_seqs):
    kv_len = [(7 * b) % 40 for b in range(n_seqs)]
    U.check_attention(U.Case(fmt, 2, 1, 128, 16, [min(1, n) for n in kv_len], kv_len, seed=18))
    U.check_attention(U.Case(fmt, 2, 1, 128, 16, [min(b % 3, n) for b, n in enumerate(kv_len)], kv_len, seed=19))


@pytest.mark.parametrize("fmt,d", SHAPES)
def test_items_that_follow_each_other_keep_their_sums(fmt, d):
    """Ten and more short items to a pair of SMs, one straight after the other: each row's weights are summed from
    two halves, whose exchange the next item's must not overtake."""
    new = [1 + b % 5 for b in range(400)]
    case = U.Case(fmt, 4, 2, d, 16, new, [n + (3 * b) % 7 for b, n in enumerate(new)], seed=30)
    kv = case.handle()
    c, batch, q = case.filled(kv), case.batch(), case.q.cuda()
    out, lse = U.check_attention(case, kv=kv, cache=c, q=q)
    for _ in range(30):
        out2, lse2 = kv.attention(c, batch, q)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
@pytest.mark.parametrize("at", [0, 64, 200, 290])
def test_values_of_far_apart_sizes(fmt, d, window, sinks, at):
    """A value 2^40 above the others counts for the rows that see it alone, in whichever key tile it is."""
    case = U.Case(fmt, 4, 2, d, 32, [300, 40, 1], [300, 291, 291], seed=31)
    for v in case.v:
        v[:] *= 2.0 ** -30
        if at < len(v):
            v[at] *= 2.0 ** 40
    U.check_attention(case, window, sinks)


@pytest.mark.parametrize("d", [128, 256, 512])
def test_values_of_far_apart_sizes_in_whole_items(d):
    """The same in more items than there are pairs of SMs, which are then not cut: one after the other, with
    their large value in another tile, or in none."""
    case = U.Case("e4m3", 2, 2, d, 16, [140] * 60, [140 + 9 * (b % 7) for b in range(60)], seed=32)
    for b, v in enumerate(case.v):
        if b % 5:
            v[(37 * b) % 140] *= 2.0 ** (40 if b % 2 else -40)
    U.check_attention(case)


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
def test_hidden_values_and_far_apart_sizes(fmt, d, window, sinks):
    """NaN and infinities among values of far apart sizes change only the rows that see them."""
    case = U.Case(fmt, 2, 1, d, 16, [90, 1], [150, 200], seed=40)
    case.v[0][20] *= 2.0 ** 40
    case.v[0][140] *= 2.0 ** 50
    case.v[0][130, 0, 5] = math.nan
    case.v[0][100, 0, d - 1] = math.inf
    case.k[0][145, 0, 3] = math.nan
    case.v[0][30, 0, 40] = math.nan
    case.k[1][20, 0, 3] = math.nan
    case.v[1][60] = 0
    U.check_attention(case, window, sinks)


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("e4m3", 256)])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 1, 9]])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 40, 2 ** 40), (5, 2 ** 31 - 1)])
def test_windows_and_sinks_as_long_as_numbers_go(fmt, d, new, window, sinks):
    case = U.Case(fmt, 4, 2, d, 32, new, [300, 40, 5], seed=41)  # (four rows before the first position)
    kv = case.handle()
    c, q = case.filled(kv), case.q.cuda()
    out, lse = kv.attention(c, case.batch(), q, window=window, sinks=sinks)
    _ok(kv)
    want, wl, tol, ltol = U.attention(case)
    U.check_close(lse, wl, ltol, "lse")
    U.check_close(out, want, tol, "out")


@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("new", [1, 160])
@pytest.mark.parametrize("big,score", [(2.0 ** 40, -45.0), (0.0, 30.0), (2.0 ** -40, 25.0)])
def test_values_far_from_their_weights(d, new, big, score):
    """A large value of hardly any weight, and zeros or small ones of nearly all: the other keys' share of the
    output is as exact as their own sizes ask for."""
    for at in (3, 150, 299 - new // 2):
        case = U.Case("e4m3", 2, 1, d, 64, [new], [300], seed=33)
        u = torch.randn(d, generator=torch.Generator().manual_seed(d)).to(torch.bfloat16)
        case.q[:] = u
        case.k[0][:] *= 0.25
        case.k[0][at, 0] = (u.double() * score * d ** 0.5 / (u.double() ** 2).sum()).to(torch.bfloat16)
        case.v[0][at] *= big
        U.check_attention(case)


@pytest.mark.parametrize("fmt,hq,hkv,d", [("bf16", 18, 2, 128), ("e4m3", 16, 1, 256), ("bf16", 33, 1, 256),
                                          ("e4m3", 64, 1, 128), ("bf16", 64, 1, 512), ("e4m3", 66, 2, 512)])
@pytest.mark.parametrize("new", [[1, 1, 1], [4, 1, 9]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1024, 4)])
def test_many_heads_per_kv_head_over_long_caches(fmt, hq, hkv, d, new, window, sinks):
    case, h, c, want = _large(fmt, hq, hkv, d, 32, new, [6001, 700, 2048], seed=22)
    out, lse = h.attention(c, case.batch(), case.q.cuda(), window=window, sinks=sinks)
    _ok(h)
    w, wl = want(window, sinks)
    # As for other long caches: a rounding of the weights, one of the result, and what is held in fp32.
    U.check_close(lse, wl, torch.full_like(wl, 2.0 ** -10), "lse")
    U.check_close(out, w, 2 * U.BF * w.abs() + U.BF + 2.0 ** -10, "out")


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("new,max_new", [([1, 1, 1], 50), ([1, 0, 1], 2), ([30, 1, 3], 1000)])
def test_a_bound_above_the_longest_sequence(fmt, d, new, max_new):
    case = U.Case(fmt, 4, 2, d, 32, new, [300, 40, 131], seed=23)
    kv = case.handle()
    c, b = case.filled(kv), case.batch()
    out, lse = kv.attention(c, B.KVBatch(*b.tensors, max_new=max_new), case.q.cuda())
    _ok(kv)
    want, wl, tol, ltol = U.attention(case)
    U.check_close(lse, wl, ltol, "lse")
    U.check_close(out, want, tol, "out")


def test_shares_past_32_bits():
    """More key tiles than 32-bit arithmetic divides among the CTAs: 520 single tokens on 131072, whose tables
    name the same 64 pages over and over, so that each sees the same 1024 keys 128 times."""
    n, hq, d, times = 520, 8, 128, 128
    kv = B.PagedKV(hq, hq, d, 16, 64, "bf16", max_tokens=1024, max_seqs=n)
    c = kv.new_cache()
    g = torch.Generator(device="cuda").manual_seed(24)
    c.k.normal_(generator=g)
    c.v.normal_(generator=g)
    q = torch.randn(n, hq, d, generator=g, device="cuda").bfloat16()
    pages = torch.arange(64, dtype=torch.int32, device="cuda").repeat(n, times)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out, lse = kv.attention(c, B.KVBatch(cu, torch.full_like(cu[:-1], 1024 * times), pages, max_new=1), q)
    _ok(kv)
    k, v = (t.transpose(1, 2).reshape(1024, hq, d).double() for t in (c.k, c.v))
    s = torch.einsum("thd,jhd->thj", q.double(), k) * d ** -0.5
    want = torch.einsum("thj,jhd->thd", torch.softmax(s, -1), v)
    # Sums of 2^17 terms in fp32, in pieces of at most 2^17: 2^-7 at worst, of the weights and of the values.
    U.check_close(lse, (torch.logsumexp(s, -1) + math.log(times)).cpu(), torch.full((n, hq), 2.0 ** -7 + 2.0 ** -10).double(), "lse")
    U.check_close(out, want.cpu(), (2 * U.BF * want.abs() + U.BF + 2.0 ** -6).cpu(), "out")


@pytest.mark.parametrize("fmt,page,pages", [("bf16", 128, 20000), ("e4m3", 16, 300000)])
def test_offsets_beyond_32_bits(fmt, page, pages):
    """The sequence's pages are the last of a cache of over 2^32 bytes."""
    case = U.Case(fmt, 4, 2, 512, page, [1, 40], [300, 200], seed=20)
    case.pages[case.pages >= 0] += pages - case.n_pages
    case.n_pages = pages
    assert 2 * pages * page * 512 * (2 if fmt == "bf16" else 1) > 1 << 32
    case.garbage = "zero"
    kv = case.handle()
    c = case.filled(kv)
    U.check_attention(case, kv=kv, cache=c)
    one = U.Case(fmt, 4, 2, 512, page, [1, 1], [300, 200], seed=20)
    one.pages, one.n_pages = case.pages, pages
    U.check_attention(one, kv=kv, cache=c)
    k, _ = kv.read(c, case.batch([300, 200]), n_tokens=500)
    want = torch.cat([case.stored("k", b) for b in range(2)])
    U.check_close(k, want, (U.BF + U.F32) * want.abs(), "k")


def test_expanded_inputs():
    """Queries and keys that are one row seen many times (strides of 0)."""
    case = U.Case("bf16", 4, 2, 128, 16, [20], [20], seed=21)
    case.q[:] = case.q[:1, :1]
    case.k[0][:] = case.k[0][:1]
    kv = case.handle()
    c = case.empty_cache(kv)
    kv.write(c, case.batch(), case.k[0][:1].cuda().expand(20, -1, -1), case.v[0].cuda())
    U.check_attention(case, kv=kv, cache=c, q=case.q[:1, :1].cuda().expand(20, 4, -1))


@pytest.mark.parametrize("layer,fmt", [("sliding", "e4m3"), ("global", "bf16")])
def test_example_serves_a_layer(layer, fmt):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layer.py")
    spec = importlib.util.spec_from_file_location("serve_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off, status = m.main(["--layer", layer, "--format", fmt, "--users", "4", "--steps", "3"])
    # Two ways of cutting the same sums: bf16 outputs of each stage, a few roundings apart (a token near a
    # tie of the router may change an expert, which the norm over all tokens bounds).
    assert status == 0 and off < 2e-2


def test_captured_step_replays_with_new_lengths():
    """Write and attention of a decode step in a graph; the batch's tensors change between replays."""
    case = U.Case("e4m3", 4, 2, 256, 16, [1, 1], [30, 51], seed=11)
    kv = case.handle()
    batch = case.batch()
    q = case.q.cuda()
    k = torch.stack([case.k[b][-1] for b in range(2)]).cuda()
    v = torch.stack([case.v[b][-1] for b in range(2)]).cuda()
    c = case.filled(kv)
    kv.write(c, batch, k, v)
    want, wlse = kv.attention(c, batch, q)
    torch.cuda.synchronize()
    c2 = case.filled(kv)
    for b in range(2):
        page, slot = int(case.pages[b, (case.kv[b] - 1) // 16]), (case.kv[b] - 1) % 16
        c2.v.view(torch.uint8)[page, :, slot] = 0
    batch.tensors[1].fill_(1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.write(c2, batch, k, v)
        out, lse = kv.attention(c2, batch, q)
    batch.tensors[1].copy_(torch.tensor(case.kv, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    _ok(kv)


def test_calls_on_two_streams_are_ordered():
    case = U.Case("bf16", 4, 2, 256, 16, [64], [640], seed=12)
    kv = case.handle()
    c = case.filled(kv)
    q = case.q.cuda()
    want, _ = kv.attention(c, case.batch(), q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    batch = case.batch()
    for _ in range(4):
        c2 = case.filled(kv)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got, _ = kv.attention(c2, batch, q)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)


@pytest.mark.parametrize("new", [1, 150])
def test_calls_of_one_handle_on_two_streams_follow_each_other(new):
    """The handle's workspace holds pieces of cut items: with nothing ordered by hand, a call on one stream starts
    after the other stream's, long and short ones in turn."""
    cases = [U.Case("bf16", 16, 2, 512, 64, [new], [n], seed=n) for n in (60000, 3000, 20000)]
    for case in cases:
        case.n_pages = max(x.n_pages for x in cases)
    kv = cases[0].handle()
    calls = [(case.filled(kv), case.batch(), case.q.cuda()) for case in cases]
    want = [kv.attention(*call) for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(24):
        with torch.cuda.stream(streams[i % 2]):
            got.append(kv.attention(*calls[i % 3]))
    torch.cuda.synchronize()
    _ok(kv)
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 3][0]) and torch.equal(lse, want[i % 3][1]), i


def test_a_dropped_handle_leaves_its_workspace_to_the_stream_that_uses_it():
    case = U.Case("bf16", 4, 2, 256, 16, [200], [3000], seed=36)
    kv = case.handle()
    c, batch, q = case.filled(kv), case.batch(), case.q.cuda()
    want, _ = kv.attention(c, batch, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    at, nbytes = kv.workspace.data_ptr(), kv.nbytes
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        out, _ = kv.attention(c, batch, q)
    del kv
    other = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert all(t.data_ptr() != at for t in other)
    for t in other:
        t.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("new", [1, 200])
def test_a_workspace_of_memory_still_being_written(new):
    """Made on a side stream, from a block that work queued there before still writes."""
    case = U.Case("bf16", 4, 2, 256, 16, [new], [3000], seed=37)
    kv = case.handle()
    c, batch, q = case.filled(kv), case.batch(), case.q.cuda()
    want, _ = kv.attention(c, batch, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block = torch.empty(kv.nbytes, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        block.fill_(255)
        at = block.data_ptr()
        del block
        late = case.handle()
        assert late.workspace.data_ptr() == at
        out, _ = late.attention(c, batch, q)
    torch.cuda.synchronize()
    assert late.status() == (B.MOE_FFN_OK, 0)
    assert torch.equal(out, want)


def test_bad_tables_set_the_status_word():
    """Page ids and lengths out of range: nothing out of the cache is touched, and the status says so."""
    case = U.Case("bf16", 4, 2, 256, 16, [1, 1, 20], [40, 20, 33], seed=13)
    kv = case.handle()
    c = case.filled(kv)
    for change in ("page", "negative", "kv_len", "cu_q"):
        batch = case.batch()
        cu, kv_len, pages = batch.tensors
        if change == "page":
            pages[1, 0] = case.n_pages
        elif change == "negative":
            pages[1, 1] = -1
        elif change == "kv_len":
            kv_len[1] = pages.shape[1] * 16 + 1
        else:
            cu[2] = 40
        out, _ = kv.attention(c, batch, case.q.cuda())
        torch.cuda.synchronize()
        assert kv.status() == (B.MOE_FFN_EDEVICE, B.STATUS_BITS["BAD_INDEX"]), change
        kv.read(c, batch, n_tokens=case.T)
        assert kv.status()[1] in (0, B.STATUS_BITS["BAD_INDEX"])
    want, _ = U.check_attention(case, kv=kv, cache=c)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1], [3, 20]])
def test_rows_before_the_first_sequence(fmt, new):
    """cu_q must start at 0: the status word says so, and the rows before it are rows of no sequence."""
    case = U.Case(fmt, 4, 2, 256, 16, new, [40, 33], seed=34, pad_rows=4)
    kv = case.handle()
    c = case.filled(kv)
    batch = case.batch()
    batch.tensors[0].add_(3)
    q = case.q.cuda()
    out, lse = kv.attention(c, batch, q, out=torch.ones_like(q))
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_EDEVICE, B.STATUS_BITS["BAD_INDEX"])
    for rows in (slice(0, 3), slice(case.T - 1, case.T)):
        assert not out[rows].any() and (lse[rows] == -math.inf).all()
    for call in (lambda: kv.read(c, batch, n_tokens=case.T),
                 lambda: kv.write(kv.new_cache(), batch, q[:, :2], q[:, 2:])):
        call()
        torch.cuda.synchronize()
        assert kv.status() == (B.MOE_FFN_EDEVICE, B.STATUS_BITS["BAD_INDEX"])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 30, 20]])
@pytest.mark.parametrize("bad", [-1, -2, -7, -2 ** 31, "n_pages", 2 ** 31 - 1])
def test_every_bad_page_id_is_reported(fmt, new, bad):
    """By each operator that needs it; the other sequences do not notice."""
    case = U.Case(fmt, 4, 2, 256, 16, new, [40, 50, 33], seed=35)
    kv = case.handle()
    c = case.filled(kv)
    q = case.q.cuda()
    want, _ = kv.attention(c, case.batch(), q)
    batch = case.batch()
    batch.tensors[2][1, 3] = case.n_pages if bad == "n_pages" else bad  # of positions 48 and 49
    out, _ = kv.attention(c, batch, q)
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_EDEVICE, B.STATUS_BITS["BAD_INDEX"])
    a, b = case.cu[1], case.cu[2]
    assert torch.equal(out[:a], want[:a]) and torch.equal(out[b:], want[b:])
    for call in (lambda: kv.read(c, batch, n_tokens=case.T),
                 lambda: kv.write(c, batch, q[:, :2], q[:, 2:])):
        call()
        torch.cuda.synchronize()
        assert kv.status() == (B.MOE_FFN_EDEVICE, B.STATUS_BITS["BAD_INDEX"])
    # An entry that no token sees may hold anything.
    batch.tensors[2][1, 3] = case.pages[1, 3]
    batch.tensors[2][2, 3] = -2 if bad == "n_pages" else bad
    kv.attention(c, batch, q)
    _ok(kv)


def test_no_report_is_lost_between_calls():
    """On a stream that does not wait for the legacy one: each bad call is reported, right after the last report."""
    case = U.Case("bf16", 2, 2, 128, 16, [1], [20], seed=38)
    kv = case.handle()
    c, batch, q = case.filled(kv), case.batch(), case.q.cuda()
    batch.tensors[2][0, 1] = -1
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(200):
            kv.attention(c, batch, q)
            assert kv.status() == (B.MOE_FFN_EDEVICE, B.STATUS_BITS["BAD_INDEX"])
        assert kv.status() == (B.MOE_FFN_OK, 0)


def test_empty_batches_do_nothing():
    case = U.Case("bf16", 4, 2, 256, 16, [], [], seed=14)
    kv = case.handle()
    c = kv.new_cache()
    x = torch.zeros(0, 2, 256, dtype=torch.bfloat16, device="cuda")
    kv.write(c, case.batch(), x, x)
    out, lse = kv.attention(c, case.batch(), torch.zeros(0, 4, 256, dtype=torch.bfloat16, device="cuda"))
    assert out.shape == (0, 4, 256) and lse.shape == (0, 4)
    # Rows but no sequences: all padding.
    out, lse = kv.attention(c, case.batch(), torch.ones(1, 4, 256, dtype=torch.bfloat16, device="cuda"))
    _ok(kv)
    assert not out.any() and torch.isinf(lse).all()


def test_caches_of_another_kind_of_layer_are_refused():
    sliding, glob = B.PagedKV(16, 8, 256, 64, 6), B.PagedKV(16, 2, 512, 64, 6)
    e4m3, same = B.PagedKV(16, 8, 256, 64, 6, "e4m3"), B.PagedKV(32, 8, 256, 64, 6, max_seqs=3)
    c = sliding.new_cache()
    cu, kv_len = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, 3], [3]))
    batch = B.KVBatch(cu, kv_len, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), max_new=3)
    x = {h: torch.ones(3, h.kv_heads, h.head_dim, dtype=torch.bfloat16, device="cuda") for h in (sliding, glob, e4m3, same)}
    for h, other in ((glob, c), (e4m3, c), (sliding, glob.new_cache()), (sliding, e4m3.new_cache()),
                     (glob, B.KVCache(c.k, c.v))):
        for call in (lambda: h.write(other, batch, x[h], x[h]), lambda: h.read(other, batch, 3),
                     lambda: h.attention(other, batch, x[h].repeat_interleave(h.q_heads // h.kv_heads, 1))):
            with pytest.raises(ValueError):
                call()
    assert not c.k.any() and not c.v.any()
    # Another handle of the same shape may use it, and tensors put together by hand are checked per call.
    same.write(c, batch, x[same], x[same])
    k, v = sliding.read(B.KVCache(c.k, c.v), batch, 3)
    _ok(sliding)
    assert torch.equal(k, x[same]) and torch.equal(v, x[same])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_outputs_that_overlap_what_is_read_are_refused(fmt):
    case = U.Case(fmt, 4, 2, 256, 16, [2], [40], seed=39)
    kv = case.handle()
    c, batch = case.filled(kv), case.batch()
    q = torch.zeros(64, 4, 256, dtype=torch.bfloat16, device="cuda")[:2]
    out, lse = torch.empty(2, 4, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 4, device="cuda")
    kept = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]
    rows, struct = kv._rows("q", q, 4), batch.of(2)
    inside = [t.data_ptr() + 64 for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]

    def attention(o, l):
        return B.moe_ffn_kv_attention(kv.ctx, c.struct, struct, rows, 0.1, 0, 0, o, l, 0)

    assert attention(out.data_ptr(), q.data_ptr()) == B.MOE_FFN_EINVAL
    for at in inside:
        assert attention(at, lse.data_ptr()) == B.MOE_FFN_EINVAL
        assert attention(out.data_ptr(), at) == B.MOE_FFN_EINVAL
        assert B.moe_ffn_kv_read(kv.ctx, c.struct, struct, at, out.data_ptr(), 0) == B.MOE_FFN_EINVAL
        assert B.moe_ffn_kv_read(kv.ctx, c.struct, struct, out.data_ptr(), at, 0) == B.MOE_FFN_EINVAL
    assert attention(out.data_ptr(), lse.data_ptr()) == B.MOE_FFN_OK
    _ok(kv)
    for t, was in zip((c.k, c.v, c.k_scale, c.v_scale), kept):
        assert torch.equal(t.view(torch.uint8), was.view(torch.uint8))


def test_refusals():
    case = U.Case("bf16", 4, 2, 256, 16, [2], [5], seed=15)
    kv = case.handle()
    c, batch, q = case.filled(kv), case.batch(), case.q.cuda()
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=math.inf), dict(scale=-1.0)):
        with pytest.raises(B.MoeFFNError) as e:
            kv.attention(c, batch, q, **kw)
        assert e.value.status == B.MOE_FFN_EINVAL
    with pytest.raises(B.MoeFFNError) as e:
        kv.attention(c, batch, q, out=q)
    assert e.value.status == B.MOE_FFN_EINVAL
    big = torch.zeros(kv.cfg.max_tokens + 1, 4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.MoeFFNError) as e:
        kv.attention(c, batch, big)
    assert e.value.status == B.MOE_FFN_ETOOBIG
    flat = torch.zeros(4 * 256 * 2 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.MoeFFNError) as e:
        kv.attention(c, batch, flat[4:].view(2, 4, 256))
    assert e.value.status == B.MOE_FFN_EALIGN
    with pytest.raises(ValueError, match="multiples of 8"):
        kv.attention(c, batch, torch.zeros(2, 4, 257, dtype=torch.bfloat16, device="cuda")[:, :, :256])
    L = B.lib()
    rows = kv._rows("q", q, 4)
    st = batch.struct
    st.n_tokens = 2
    args = (rows, 0.1, 0, 0, q.data_ptr() + (1 << 20), None, None)
    assert L.moe_ffn_kv_attention(kv._handle, B.moe_ffn_kv_cache(), st, *args) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_attention(kv._handle, c.struct, st, rows, 0.1, 0, 0, None, None, None) == B.MOE_FFN_EINVAL
    st.n_seqs = kv.cfg.max_seqs + 1
    assert L.moe_ffn_kv_attention(kv._handle, c.struct, st, *args) == B.MOE_FFN_ETOOBIG
    st.n_seqs = 1
    st.pages_stride = 0
    assert L.moe_ffn_kv_attention(kv._handle, c.struct, st, *args) == B.MOE_FFN_EINVAL
