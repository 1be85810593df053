"""The beam search's selection on a GB300 against its definition in 64 bits: beams and tokens are equal, scores
are off by half a step of fp32 (2^-24) and the 1e-7 that the sums are held to."""
import math

import pytest
import torch

from mixture_experts_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def _wanted(logits, scores, count, finished=None, end=0):
    U, K = scores.shape
    x = logits.reshape(U, K, -1).double()
    V = x.shape[-1]
    x = torch.log_softmax(x, -1)
    if finished is not None:
        one = torch.full((V,), -math.inf, dtype=torch.float64, device=x.device)
        one[end] = 0.0
        x = torch.where(finished[..., None], one, x)
    x = (x + scores.double()[..., None]).view(U, K * V)
    x = torch.where(x > -math.inf, x, -math.inf)  # NaN is none
    best, at = torch.sort(x, dim=1, descending=True, stable=True)
    best, at = best[:, :count], at[:, :count]
    short = count - best.shape[1]
    if short > 0:
        best = torch.cat((best, torch.full((U, short), -math.inf, device=x.device, dtype=torch.float64)), 1)
        at = torch.cat((at, torch.zeros(U, short, dtype=at.dtype, device=x.device)), 1)
    none = best == -math.inf
    return best, (at // V).masked_fill(none, -1).int(), (at % V).masked_fill(none, -1).int()


def _check(logits, scores, count, finished=None, end=0, search=None, vocab=None):
    U, K = scores.shape
    search = search or B.BeamSearch(U, K, logits.shape[-1], count)
    got = search.select(logits, scores, finished=finished, end_token=end)
    torch.cuda.synchronize()
    want = _wanted(logits, scores, count, finished, end)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    inf = torch.isinf(want[0])
    assert torch.equal(torch.isinf(got[0]), inf)
    off = (got[0].double() - want[0]).abs() - 2.0 ** -24 * want[0].abs() - 1e-7
    assert inf.all() or off[~inf].max() <= 0
    return got


def _inputs(U, K, V, seed=0, dtype=torch.bfloat16, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(U * K, V, generator=g, device="cuda") * spread
    return x.to(dtype), -6 * torch.rand(U, K, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("U,K,V,C", [(1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 16), (3, 4, 1000, 8), (1, 4, 32001, 8), (5, 2, 8191, 4),
                                     (2, 5, 8193, 10), (1, 64, 777, 64), (70, 1, 501, 3), (2, 8, 262144, 16),
                                     (1, 1, 262144, 64), (1, 2, 1500000, 5)])
def test_sizes(U, K, V, C, dtype):
    logits, scores = _inputs(U, K, V, seed=U + K + V, dtype=dtype)
    _check(logits, scores, C)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spread", [0.0, 0.01, 1.0, 30.0, 1000.0])
def test_spreads(dtype, spread):
    """From rows of one value, where the lowest tokens win, to rows of which one token holds all the weight."""
    logits, scores = _inputs(2, 3, 40000, seed=int(spread) + 9, dtype=dtype, spread=spread)
    _check(logits, scores, 12)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lift", [10.0, 40.0, 1e4, 1e9])
def test_one_far_above_the_rest(dtype, lift):
    for U, K, V, C in ((2, 4, 128256, 16), (1, 3, 262144, 1), (1, 12, 50001, 22)):
        logits, scores = _inputs(U, K, V, seed=C, dtype=dtype)
        logits[torch.arange(U * K), torch.arange(U * K) * 37 % V] = lift
        _check(logits, scores, C)
        logits[::2, V - 1] = 0.75 * lift
        _check(logits, scores, C)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("count", [1, 7, 64])
def test_orders_that_fill_the_list(dtype, count):
    """Logits that ascend (each tile's are above all before), descend, or are mostly equal."""
    V = 120000
    up = torch.linspace(-400, 500, V, device="cuda")
    steps = torch.floor(up / 100)
    two = torch.where(torch.arange(V, device="cuda") % 3 == 0, 1.0, 2.0)
    logits = torch.stack((up, up.flip(0), steps, two, torch.zeros_like(up), -torch.zeros_like(up))).to(dtype)
    scores = torch.tensor([[0.0, -0.5], [-1.0, -1.0], [-2.0, -2.0]], device="cuda")
    _check(logits, scores, count)


def test_ties():
    """Equal beams: the lower beam first, then the lower token; zeros of either sign are equal."""
    g = torch.Generator(device="cuda").manual_seed(4)
    row = torch.randint(-8, 9, (50000,), generator=g, device="cuda").float()
    logits = row.to(torch.bfloat16).expand(4, 50000).contiguous()
    _check(logits, torch.full((1, 4), -1.5, device="cuda"), 64)
    # Rows of odd lengths begin at any address, and equal ones are equal all the same.
    for dtype in (torch.bfloat16, torch.float32):
        odd = (row[:49999] / 3).to(dtype).expand(7, 49999).contiguous()
        _check(odd, torch.full((1, 7), -1.5, device="cuda"), 64)
    z = torch.zeros(2, 20000, device="cuda")
    z[:, ::2] = -0.0
    z[:, 5000:] = -1.0
    _check(z, torch.zeros(1, 2, device="cuda"), 40)
    _check(z.to(torch.bfloat16), torch.zeros(1, 2, device="cuda"), 40)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K,V,C", [(64, 20000, 64), (8, 262144, 64), (37, 33001, 41)])
def test_many_candidates(K, V, C, dtype):
    """More parts and candidates than are compared at once: of random rows, of equal ones, of few values; one beam alone,
    one far ahead, most of them ended, few tokens allowed."""
    logits, scores = _inputs(2, K, V, seed=C, dtype=dtype)
    search = B.BeamSearch(2, K, V, C)
    _check(logits, scores, C, search=search)
    first = scores.clone()
    first[:, 1:] = -math.inf
    _check(logits, first, C, search=search)
    ahead = scores.clone()
    ahead[:, K // 2] = 50.0
    _check(logits, ahead, C, search=search)
    ended = (torch.arange(2 * K, device="cuda") % 5 != 0).view(2, K)
    _check(logits, scores, C, ended, 3, search=search)
    for share in (2e-5, 5e-4):
        g = torch.Generator(device="cuda").manual_seed(C)
        allowed = torch.rand(logits.shape, generator=g, device="cuda") < share
        _check(torch.where(allowed, logits, -math.inf), scores, C, search=search)
        _check(torch.where(allowed, logits, torch.finfo(dtype).min), scores, C, search=search)
    few = (logits[:1] * 0.7).round().expand(2 * K, V).contiguous()  # equal rows: ties over all beams
    for level in (torch.full_like(scores, -1.5), scores):
        _check(few, level, C, search=search)
        _check(torch.zeros_like(logits), level, C, search=search)


def test_first_step_and_finished_beams():
    logits, scores = _inputs(3, 4, 9000, seed=5)
    scores[:, 1:] = -math.inf
    _check(logits, scores, 8)
    logits, scores = _inputs(3, 4, 9000, seed=6)
    finished = torch.tensor([[True, False, False, True], [False] * 4, [True] * 4], device="cuda")
    logits[0] = math.nan  # a finished beam's logits are not looked at
    for end in (0, 8999, 17):
        got = _check(torch.where(torch.isnan(logits), 0, logits), scores, 8, finished, end)
        same = B.BeamSearch(3, 4, 9000, 8).select(logits, scores, finished, end)
        assert all(torch.equal(a, b) for a, b in zip(got, same))
        assert (got[1][2, 4:] == -1).all() and (got[2][2, :4] == end).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [300, 20000, 120001])
def test_masked_logits(dtype, V):
    """-infinity and the type's lowest value where a token is forbidden, up to all of them."""
    low = torch.finfo(dtype).min
    for value in (-math.inf, low):
        logits, scores = _inputs(2, 3, V, seed=V, dtype=dtype)
        g = torch.Generator(device="cuda").manual_seed(7)
        forbidden = torch.rand(logits.shape, generator=g, device="cuda") < 0.999
        forbidden[1] = True
        forbidden[1, V // 2] = False
        forbidden[2] = True
        forbidden[3, : V - 2] = True
        logits[forbidden] = value
        if value == low:
            # What 64 bits leave of low + log V is low.
            _check(torch.cat((logits[:2], logits[3:4])).contiguous(), scores[:1].contiguous(), 2)
            rows = logits[2:3].contiguous()
            out = B.BeamSearch(1, 1, V, 5).select(rows, torch.zeros(1, 1, device="cuda"))
            assert (out[2] == torch.arange(5, device="cuda")).all() and (out[0] + math.log(V)).abs().max() < 1e-5
        else:
            _check(logits, scores, 10)


def test_a_beam_with_nan_or_infinity_has_no_continuations():
    logits, scores = _inputs(1, 3, 30000, seed=8)
    logits[0, 29999] = math.nan
    logits[2, 5] = math.inf
    got = _check(logits, scores, 6)
    assert (got[1] == 1).all()
    scores[0, 1] = math.nan
    got = _check(logits, scores, 6)
    assert (got[1] == -1).all() and (got[0] == -math.inf).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_any_address(dtype):
    wide = torch.full((6, 5023), 99.0, dtype=dtype, device="cuda")
    for shift in range(9):
        logits, scores = _inputs(2, 3, 5003, seed=shift, dtype=dtype)
        view = wide[:, shift:shift + 5003]
        view.copy_(logits)
        search = B.BeamSearch(2, 3, 5003, 7)
        got = search.select(view, scores)
        want = _check(logits, scores, 7)
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        wide.fill_(99.0)
    one = _inputs(1, 1, 5003, seed=1, dtype=dtype)[0].expand(6, 5003)
    _check(one, torch.arange(6.0, device="cuda").view(2, 3), 7)


def test_three_dimensions_and_steps():
    logits, scores = _inputs(4, 3, 700, seed=9)
    search = B.BeamSearch(4, 3, 700, 6)
    a = search.select(logits, scores)
    b = search.select(logits.view(4, 3, 700), scores)
    wide = torch.zeros(4, 3, 2, 700, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1] = logits.view(4, 3, 700)
    c = search.select(wide[:, :, 1], scores)
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_captured_and_on_other_streams():
    logits, scores = _inputs(2, 4, 50000, seed=10)
    other, other_scores = _inputs(2, 4, 50000, seed=11)
    search = B.BeamSearch(2, 4, 50000, 8)
    want, later = (B.BeamSearch(2, 4, 50000, 8).select(a, b) for a, b in ((logits, scores), (other, other_scores)))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(9):
        with torch.cuda.stream(streams[i % 3]):
            got.append(search.select(*((logits, scores) if i % 2 == 0 else (other, other_scores))))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = search.select(logits, scores)
    logits.copy_(other)
    scores.copy_(other_scores)
    graph.replay()
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want if i % 2 == 0 else later))
    assert all(torch.equal(x, y) for x, y in zip(held, later))


def test_refusals():
    for sizes in ((-1, 4, 100, 8), (4097, 4, 100, 8), (2, 0, 100, 8), (2, 65, 100, 8), (2, 4, 0, 8), (2, 4, (1 << 24) + 1, 8),
                  (2, 4, 100, 0), (2, 4, 100, 65)):
        with pytest.raises(ValueError, match="invalid"):
            B.BeamSearch(*sizes)
    search = B.BeamSearch(2, 4, 100, 8)
    logits, scores = _inputs(2, 4, 100)
    for args, match in (((logits.half(), scores), "bfloat16"), ((logits[:7], scores), "shape"), ((logits.T.contiguous().T, scores), "rows"),
                        ((logits, scores.double()), "scores"), ((logits, scores.T.contiguous().T), "scores"),
                        ((logits, scores, scores), "finished"), ((logits, scores.cpu()), "scores must be on"),
                        ((torch.zeros(4, 2, 100, device="cuda", dtype=torch.bfloat16).transpose(0, 1), scores), "one stride")):
        with pytest.raises(ValueError, match=match):
            search.select(*args)
    done = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    for end in (-1, 100):
        with pytest.raises(B.MoeFFNError):
            search.select(logits, scores, done, end)
    empty = B.BeamSearch(0, 4, 100, 8).select(logits[:0], scores[:0])
    assert all(t.shape == (0, 8) for t in empty)


def test_rows_past_32_bits():
    U, K, V, C = 13, 10, 1 << 24, 6
    logits = torch.zeros(U * K, V, dtype=torch.bfloat16, device="cuda")  # 2.2e9 logits
    g = torch.Generator().manual_seed(4)
    rows = torch.arange(U * K).repeat_interleave(3)
    places = (torch.randint(0, V // 3, (U * K, 3), generator=g) + torch.arange(3) * (V // 3)).view(-1)
    places[-1] = V - 1
    values = (torch.rand(U * K * 3, generator=g) * 8 + 1).to(torch.bfloat16)
    logits[rows.cuda(), places.cuda()] = values.cuda()
    scores = -torch.rand(U, K, generator=g)
    got = B.BeamSearch(U, K, V, C).select(logits, scores.cuda())
    x = values.double().view(U * K, 3)
    x = x - (V - 3 + x.exp().sum(1, keepdim=True)).log() + scores.double().view(-1, 1)
    beams = torch.arange(K).repeat_interleave(3)
    for u in range(U):
        mine, token = x[u * K:(u + 1) * K].reshape(-1), places.view(U, -1)[u]
        order = sorted(range(3 * K), key=lambda i: (-float(mine[i]), int(beams[i]), int(token[i])))[:C]
        assert got[1][u].tolist() == beams[order].tolist() and got[2][u].tolist() == token[order].tolist()
        assert ((got[0][u].cpu().double() - mine[order]).abs() <= 2.0 ** -24 * mine[order].abs() + 1e-7).all()


def test_two_searches_at_once():
    # Objects of their own, on streams of their own.
    both = []
    for seed in (1, 2):
        logits, scores = _inputs(8, 5, 50_001, seed=seed)
        both.append((B.BeamSearch(8, 5, 50_001, 10), torch.cuda.Stream(), logits, scores))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for search, stream, logits, scores in both:
            with torch.cuda.stream(stream):
                got.append(search.select(logits, scores))
    torch.cuda.synchronize()
    for i, (_, _, logits, scores) in enumerate(both):
        want = _wanted(logits, scores, 10)
        for g in got[i::2]:
            assert torch.equal(g[1], want[1]) and torch.equal(g[2], want[2])


def test_a_search_made_while_its_memory_is_written():
    """Its workspace was another tensor's, which work queued on the stream it is made on still writes; the first call
    comes on another stream."""
    logits, scores = _inputs(8, 5, 50_001, seed=3)
    want = B.BeamSearch(8, 5, 50_001, 10).select(logits, scores)
    nbytes = B.moe_ffn_beam_workspace_bytes(8, 5, 50_001, 10)
    before, after = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(before):
        large = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
        was = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(before):
        for i in range(40):
            large.fill_(i)
            was.fill_(0x7f)
        del was
        search = B.BeamSearch(8, 5, 50_001, 10)
    with torch.cuda.stream(after):
        got = search.select(logits, scores)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [4000, 60001])
@pytest.mark.parametrize("count,large", [(1, 2), (1, 3), (2, 2), (1, 12), (5, 14)])
def test_few_large_logits_weigh_exactly(dtype, V, count, large):
    """Pairs of beams whose best values lie 2e-8 to 6e-8 apart. A few logits carry the weight of a row: their terms are
    good to 2^-30 of the sum (1e-9, of each of the two rows). The others weigh less than 60000 e^-30, 6e-9, of which 2^-22
    is nothing. So the order is the exact one."""
    U = 200
    g = torch.Generator().manual_seed(V + count + large)
    x = (-30 - 8 * torch.rand(U * 2, V, generator=g)).to(dtype)
    at = torch.rand(U * 2, V, generator=g).argsort(1)[:, :large]
    x.scatter_(1, at, (-2.5 * torch.rand(U * 2, large, generator=g)).to(dtype))
    x[torch.arange(U * 2), at[:, 0]] = 0
    lse = torch.logsumexp(x.double(), -1).view(U, 2)
    # The first beam's score in steps of 2^-30, so that of many the second's can be rounded near any distance.
    first = torch.rand(U, 4096, generator=g) / 64
    gap = (2e-8 + 4e-8 * torch.rand(U, 1, generator=g).double()) * (torch.arange(U) % 2 * 2 - 1).view(U, 1)
    second = (first.double() - lse[:, :1] + lse[:, 1:] + gap).float()
    found = second.double() - lse[:, 1:] - (first.double() - lse[:, :1])
    best = (found - gap).abs().argmin(1, keepdim=True)
    assert (found.gather(1, best) - gap).abs().max() < 2e-9
    scores = torch.cat((first.gather(1, best), second.gather(1, best)), 1)
    _check(x.cuda(), scores.cuda(), count)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_equal_logits_that_carry_the_weight(dtype):
    """All terms but one are off alike, by 2^-22 of each for the exponential and by half a step of the exponent, which is
    below 32 (2^-20 ln 2): together less than 2^-20."""
    V = 262_144
    far = torch.tensor([0.3, 1.7, 3.1, 5.9, 9.2, 11.3, 12.4], device="cuda").to(dtype).float()
    x = -far.view(-1, 1).expand(-1, V).clone()
    x[:, 4321] = 0.0
    scores = torch.zeros(7, 1, device="cuda")
    got = B.BeamSearch(7, 1, V, 1).select(x.to(dtype), scores)
    want = -torch.log1p((V - 1) * torch.exp(-far.double()))
    assert (got[2] == 4321).all()
    assert ((got[0][:, 0].double() - want).abs() <= 2.0 ** -20 + 2.0 ** -24 * want.abs()).all()
