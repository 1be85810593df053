"""Rotary positions on a GB300 against their definition in 64 bits.

Tolerances: the angle in half turns is rounded to fp32 (2^-25 of at most 1, times pi) and its sine and cosine are
good to two units in the last place (2^-23): together 2^-21 of either at most. In 64 bits, an angle of `a` radians is
itself known to 2^-51 a (a frequency's quotient and the product). The two products and their sum lose 3 * 2^-24 of their
magnitudes, and the result is rounded to bf16 once (2^-8)."""
import math
from fractions import Fraction

import pytest
import torch

from mixture_experts_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def _wanted(x, freqs, axes, positions, interleaved=False, scale=1.0, inverse=False):
    """(values, tolerance) of one tensor."""
    P = len(freqs)
    x = x.double().cpu()
    pos = positions.cpu().double().view(-1, x.shape[0])
    angle = torch.stack([pos[a] * f for f, a in zip(freqs, axes)], 1)[:, None]
    cos, sin = angle.cos(), angle.sin() * (-1 if inverse else 1)
    a, b = (x[..., 0:2 * P:2], x[..., 1:2 * P:2]) if interleaved else (x[..., :P], x[..., P:2 * P])
    out, tol = x.clone(), torch.zeros_like(x)
    size = (a.abs() + b.abs()) * abs(scale)
    d = size * (2.0 ** -21 + angle.abs() * 2.0 ** -51 + 3 * F32)
    u, v = scale * (a * cos - b * sin), scale * (b * cos + a * sin)
    at = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    for s, r in zip(at, (u, v)):
        out[..., s] = r
        tol[..., s] = d + BF * (r.abs() + d)
    return out, tol


def _check(got, x, *a, **kw):
    want, tol = _wanted(x, *a, **kw)
    over = (got.double().cpu() - want).abs() - tol
    assert over.max() <= 0, "off by %.3e more than allowed" % over.max()


def _freqs(P, theta=1e4):
    return [theta ** (-i / P) for i in range(P)]


def _rows(T, heads, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, heads, D, generator=g).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,P", [(1, 1, 1, 8, 4), (3, 16, 8, 256, 128), (64, 16, 2, 512, 192), (5, 12, 12, 80, 40),
                                         (7, 16, 16, 72, 36), (2, 3, 0, 64, 8), (301, 32, 8, 128, 64), (4, 2, 1, 1024, 512),
                                         (2, 5, 2, 24, 8), (3, 1024, 1, 16, 4)])
def test_widths_and_heads(T, hq, hk, D, P, interleaved):
    q, k = _rows(T, hq, D), _rows(T, hk, D, 1) if hk else None
    freqs = _freqs(P)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37 + 5
    r = B.Rotary(freqs, interleaved=interleaved)
    a, b = r.apply(q, k, pos)
    _check(a, q, freqs, [0] * P, pos, interleaved)
    if hk:
        _check(b, k, freqs, [0] * P, pos, interleaved)
    else:
        assert b is None


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [2, 3, 8])
def test_axes(axes, interleaved):
    P, T = 64, 50
    g = torch.Generator().manual_seed(axes)
    pos = torch.randint(-1000, 100000, (axes, T), generator=g, dtype=torch.int32).cuda()
    q, k = _rows(T, 4, 160), _rows(T, 2, 160, 1)
    for of in ([i * axes // P for i in range(P)], [i % axes for i in range(P)]):
        r = B.Rotary(_freqs(P), of, interleaved=interleaved, scale=1.25)
        a, b = r.apply(q, k, pos)
        for got, x in ((a, q), (b, k)):
            _check(got, x, _freqs(P), of, pos, interleaved, 1.25)
    wide = torch.full((axes, T + 9), 77, dtype=torch.int32, device="cuda")
    wide[:, :T] = pos
    assert torch.equal(r.apply(q, k, wide[:, :T])[0], a)


@pytest.mark.parametrize("first", [2 ** 31 - 300, -2 ** 31, 1_000_003, -77])
def test_far_positions(first):
    P, T = 32, 300
    q = _rows(T, 2, 64)
    pos = (torch.arange(T, dtype=torch.int64) + first).clamp(max=2 ** 31 - 1).to(torch.int32).cuda()
    freqs = _freqs(P) [:-2] + [-0.3, 12345.678]
    _check(B.Rotary(freqs).apply(q, None, pos)[0], q, freqs, [0] * P, pos)


def test_positions_of_whole_turns():
    """Frequencies that are fractions of a turn: quarters swap and negate exactly, whole turns leave all as it is."""
    q = _rows(8, 1, 16)
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    y, _ = B.Rotary([math.pi / 2] * 4 + [0.0] * 4).apply(q, None, pos * 4)
    assert torch.equal(y, q)
    y, _ = B.Rotary([math.pi / 2] * 8).apply(q, None, pos)
    assert torch.equal(y[1, 0, :8], -q[1, 0, 8:]) and torch.equal(y[2], -q[2]) and torch.equal(y[7, 0, :8], q[7, 0, 8:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_transposed_map(interleaved):
    """Back again, and the gradient: sums g . R(x) and R^T(g) . x are the same number, and differences of R's outputs
    (it is linear) are those of the transposed map's."""
    P, T = 24, 9
    freqs = _freqs(P)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1001
    r = B.Rotary(freqs, interleaved=interleaved, scale=0.75)
    x, g = _rows(T, 3, 56), _rows(T, 3, 56, 1)
    back, _ = r.apply(g, None, pos, inverse=True)
    _check(back, g, freqs, [0] * P, pos, interleaved, 0.75, inverse=True)
    y, _ = r.apply(x, None, pos)
    left, right = (g.double() * y.double()), (back.double() * x.double())
    # Half a step of each product's rounded factor.
    tol = 1.01 * BF * (left.abs().sum((1, 2)) + right.abs().sum((1, 2)))
    assert ((left.sum((1, 2)) - right.sum((1, 2))).abs() <= tol).all()
    h = torch.zeros_like(x)
    h[:, 1, 5] = 1.0
    column, _ = r.apply(h, None, pos)
    want = (column.double() * g.double()).sum((1, 2))
    assert ((back[:, 1, 5].double() - want).abs() <= 1.01 * BF * (want.abs() + (column.double() * g.double()).abs().sum((1, 2)))).all()


def test_places():
    """Views of a fused projection, transposed tensors, and in place."""
    T, freqs = 33, _freqs(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 9
    fused = _rows(T, 4 + 2 + 2, 160)
    was = fused.clone()
    q, k, v = fused.split((4, 2, 2), 1)
    r = B.Rotary(freqs)
    want = r.apply(q, k, pos)
    _check(want[0], q, freqs, [0] * 64, pos)
    assert want[0].is_contiguous() and torch.equal(fused, was)
    qt, kt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k))
    for got, w in zip(r.apply(qt, kt, pos), want):
        assert torch.equal(got, w)
    for a, b in ((qt, kt), (q, k)):
        got = r.apply(a, b, pos, inplace=True)
        assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert torch.equal(v, was[:, 6:])
    # One head's keys for all, which only a new tensor can hold turned.
    one = was[:, 4:5].expand(T, 3, 160)
    got = r.apply(was[:, :4], one, pos)[1]
    for h in range(3):
        assert torch.equal(got[:, h], want[1][:, 0])
    with pytest.raises(B.MoeFFNError):
        r.apply(was[:, :4], one, pos, inplace=True)


def test_no_tokens_and_values_that_are_not_finite():
    r = B.Rotary(_freqs(16))
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert r.apply(e, e, torch.empty(0, dtype=torch.int32, device="cuda"))[0].shape == (0, 2, 64)
    q = _rows(2, 2, 64)
    pos = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    want = r.apply(q, None, pos)[0].clone()
    q[0, 1, 3] = float("nan")
    q[1, 0, 60] = float("inf")
    got = r.apply(q, None, pos)[0]
    odd = torch.zeros(2, 2, 64, dtype=torch.bool, device="cuda")
    odd[0, 1, 3] = odd[0, 1, 19] = odd[1, 0, 60] = True
    assert torch.isnan(got[0, 1, 3]) and torch.isnan(got[0, 1, 19]) and torch.isinf(got[1, 0, 60])
    assert torch.equal(got[~odd], want[~odd])


def test_captured_and_on_another_stream():
    r = B.Rotary(_freqs(128))
    q, k = _rows(16, 16, 256), _rows(16, 8, 256, 1)
    pos = torch.arange(16, dtype=torch.int32, device="cuda")
    want = r.apply(q, k, pos)
    later = r.apply(q, k, pos + 100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = r.apply(q, k, pos)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = r.apply(q, k, pos)
    torch.cuda.synchronize()
    pos += 100
    graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i]) and torch.equal(held[i], later[i])


def test_refusals():
    r = B.Rotary(_freqs(32), [0] * 16 + [1] * 16)
    q = _rows(4, 2, 64)
    pos = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for args, match in (((q.float(), None, pos), "bfloat16"), ((q, q[:3], pos), "shape"), ((q, None, pos[0]), "positions"),
                        ((q, None, pos.long()), "positions"), ((q, None, pos[:, :3]), "positions"),
                        ((q, None, pos.cpu()), "positions must have"), ((q, _rows(4, 1, 128), pos), "k must be"),
                        ((q.transpose(1, 2).contiguous().transpose(1, 2), None, pos), None)):
        if match is None:
            with pytest.raises(ValueError):
                r.apply(*args, inplace=True)
        else:
            with pytest.raises(ValueError, match=match):
                r.apply(*args)
    with pytest.raises(B.MoeFFNError):  # 32 pairs do not fit
        r.apply(_rows(4, 2, 56), None, pos)
    x = _rows(5, 2, 64)
    with pytest.raises(B.MoeFFNError):  # each in place, but over the other
        r.apply(x[:4], x[1:], pos, inplace=True)


def test_places_past_32_bits():
    T, heads, D = 270_000, 16, 512  # 2.2e9 elements
    q = torch.empty(T, heads, D, dtype=torch.bfloat16, device="cuda").normal_()
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs = _freqs(D // 2)
    rows = torch.tensor([0, 1, 262_143, 262_144, T - 1], device="cuda")  # (2^31 elements end with row 262143)
    before = q[rows]
    B.Rotary(freqs).apply(q, None, positions, inplace=True)
    _check(q[rows], before, freqs, [0] * (D // 2), positions[rows])


def test_dropped_while_another_stream_still_turns():
    """The table's memory goes to new tensors of the stream it was made on only after the queued call."""
    T = 64
    q = _rows(T, 16, 256)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 7
    want = B.Rotary(_freqs(128)).apply(q, None, pos)[0]
    side = torch.cuda.Stream()
    large = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    r = B.Rotary(_freqs(128))
    nbytes = r.table.numel() * 8
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(40):
            large.fill_(i)
        got = r.apply(q, None, pos)[0]
    del r
    over = [torch.full((nbytes,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(200)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(over) == 200


def test_far_positions_and_fast_turns():
    """Angles of up to 10^15 radians, against their exact remainders: off by 2^-32 turns and the fp32 rounding, whatever the
    position and the frequency (together with the sine's, 2^-21 as above)."""
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
    freqs = [1.0, -0.3, 12345.678, 1e6, 333333.3, 7654321.0, 1e-3, 2.0 ** 20]
    at = [2 ** 31 - 1, -2 ** 31, 2 ** 24, 10 ** 6, -10 ** 6 - 3, 2 ** 30 + 12345, 1, 0]
    angle = torch.tensor([[float(Fraction(f) * p % two_pi) for f in freqs] for p in at], dtype=torch.float64)[:, None]
    q = _rows(len(at), 16, 16)
    got = B.Rotary(freqs).apply(q, None, torch.tensor(at, dtype=torch.int64).to(torch.int32).cuda())[0].double().cpu()
    a, b = q.double().cpu().split(8, -1)
    d = (a.abs() + b.abs()) * (2.0 ** -21 + 3 * F32)
    for r, g in ((a * angle.cos() - b * angle.sin(), got[..., :8]), (b * angle.cos() + a * angle.sin(), got[..., 8:])):
        assert ((g - r).abs() <= d + BF * (r.abs() + d)).all()
