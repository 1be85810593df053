"""block_norm on a GB300 against its formula in 64 bits.

Tolerances: a sum of H squares in fp32, in any order, is off by at most H * 2^-24 relative, its root by half that; the
products and sums around it by 2^-24 each of what they yield; y and n are rounded to bf16 once (2^-8). An error dy of y
before its rounding moves n by dy / rms(y) and by the relative error of rms(y)."""
import pytest
import torch

from mixture_experts_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def _inputs(T, H, seed=0, gate="token"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g) * 4
    x[:, ::13] *= 30
    block = torch.randn(T, H, generator=g) * torch.rand(T, 1, generator=g) * 5
    post, pre = (0.2 * torch.randn(H, generator=g) for _ in range(2))
    s = {"x": x, "block": block, "gate": None}
    if gate:
        s["gate"] = torch.randn(T if gate == "token" else 1, H, generator=g).expand(T, H)
    s = {n: t if t is None else t.to(torch.bfloat16).cuda() for n, t in s.items()}
    if gate == "one":
        s["gate"] = s["gate"][:1].expand(T, H)
    return dict(s, post=post.cuda(), pre=pre.cuda())


def _wanted(x, block=None, post=None, gate=None, scale=1.0, pre=None, eps=EPS):
    """(y, n, tolerance of y, tolerance of n)."""
    H = x.shape[1]
    x = x.double()
    b, db = torch.zeros_like(x), torch.zeros_like(x)
    if block is not None:
        b = block.double()
        if post is not None:
            b = b / (b.square().mean(-1, keepdim=True) + eps).sqrt() * (1 + post.double())
            db = b.abs() * (H / 2 + 6) * F32 + (b / (1 + post.double())).abs() * F32
        if gate is not None:
            b, db = b * gate.double(), db * gate.double().abs() + (b * gate.double()).abs() * F32
    y = scale * (x + b)
    dy = abs(scale) * (db + (x + b).abs() * 2 * F32)
    ty = dy + BF * (y.abs() + dy)
    if pre is None:
        return y, None, ty, None
    rms = (y.square().mean(-1, keepdim=True) + eps).sqrt()
    n = y / rms * (1 + pre.double())
    drms = (dy * y.abs()).mean(-1, keepdim=True) / rms ** 2
    dn = dy / rms * (1 + pre.double()).abs() + n.abs() * (drms + (H / 2 + 6) * F32) + (y / rms).abs() * F32
    return y, n, ty, dn + BF * (n.abs() + dn)


def _check(got, want, tol):
    over = (got.double() - want).abs() - tol
    assert over.max() <= 0, "off by %.3e more than allowed" % over.max()


def _run(**kw):
    y, n = B.block_norm(**kw)
    torch.cuda.synchronize()
    wy, wn, ty, tn = _wanted(**kw)
    if y is not None:
        _check(y, wy, ty)
    if n is not None:
        _check(n, wn, tn)
    return y, n


@pytest.mark.parametrize("gate", ["", "one", "token"])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 16), (5, 264), (64, 2816), (2, 4096), (3, 4104), (1, 8200), (7, 12296), (2, 16384),
                                 (1300, 40), (6, 512), (9, 520), (4001, 2816), (7000, 1800), (2800, 4096)])
def test_whole_form(T, H, gate):
    _run(**_inputs(T, H, seed=T + H, gate=gate), scale=0.8)


@pytest.mark.parametrize("T,H", [(1, 2816), (9, 72), (4100, 2816), (2900, 3592)])
def test_parts(T, H):
    s = _inputs(T, H, seed=3)
    _run(x=s["x"], pre=s["pre"])
    assert B.block_norm(s["x"], pre=s["pre"])[0] is None
    _run(x=s["x"], scale=-0.5)
    _run(x=s["x"], block=s["block"])
    _run(x=s["x"], block=s["block"], gate=s["gate"], pre=s["pre"])
    _run(x=s["x"], block=s["block"], post=s["post"], eps=0.5)
    y, n = _run(x=s["x"], block=s["block"], post=s["post"], scale=2.0)
    assert n is None
    both = B.block_norm(s["x"], s["block"], post=s["post"], scale=2.0, pre=s["pre"])
    assert torch.equal(both[0], y)


def test_rows_of_zeros_and_of_one_value():
    s = _inputs(4, 256, seed=4)
    s["block"][0] = 0
    s["x"][0] = 0
    s["block"][1] = 3.0
    s["x"][2] = 0
    y, n = _run(**s)
    assert not y[0].any() and not n[0].any()


def test_small_and_large_rows():
    s = _inputs(6, 512, seed=5)
    for i, f in enumerate((2.0 ** -60, 2.0 ** -10, 1.0, 2.0 ** 20, 2.0 ** 40)):
        s["block"][i] *= f
        s["x"][i] *= f
    _run(**s)


def test_what_is_not_finite_stays_in_its_row():
    s = _inputs(4, 320, seed=6)
    clean = B.block_norm(**s)
    s["x"][1, 7] = float("nan")
    s["block"][2, 300] = float("inf")
    y, n = B.block_norm(**s)
    for a, b in zip((y, n), clean):
        assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])
        assert torch.isnan(a[2]).any()
    assert torch.isnan(y[1, 7]) and torch.isnan(n[1]).all()


def test_strided_rows_and_places():
    s = _inputs(37, 264, seed=7)
    want = B.block_norm(**s, scale=0.7)
    wide = torch.zeros(37, 5, 264, dtype=torch.bfloat16, device="cuda")
    wide[:, 0], wide[:, 1], wide[:, 2] = s["x"], s["block"], s["gate"]
    y, n = B.block_norm(wide[:, 0], wide[:, 1], gate=wide[:, 2], post=s["post"], pre=s["pre"], scale=0.7, out=wide[:, 3],
                        normed=wide[:, 4])
    assert y.data_ptr() == wide[:, 3].data_ptr()
    for got, w in zip((y, n), want):
        assert torch.equal(got, w)
    # y over x, n over block.
    y, n = B.block_norm(wide[:, 0], wide[:, 1], gate=wide[:, 2], post=s["post"], pre=s["pre"], scale=0.7, out=wide[:, 0],
                        normed=wide[:, 1])
    assert torch.equal(wide[:, 0], want[0]) and torch.equal(wide[:, 1], want[1])
    assert torch.equal(wide[:, 2], s["gate"])


@pytest.mark.parametrize("T,H", [(9, 264), (4500, 2816)])
def test_in_place_over_many_rows(T, H):
    s = _inputs(T, H, seed=11, gate="one")
    want = B.block_norm(**s)
    y, n = B.block_norm(**s, out=s["x"], normed=s["block"])
    assert y is s["x"] and torch.equal(y, want[0]) and torch.equal(n, want[1])


def test_no_tokens():
    y, n = B.block_norm(torch.empty(0, 2816, dtype=torch.bfloat16, device="cuda"), pre=torch.zeros(2816, device="cuda"), scale=2.0)
    assert y.shape == n.shape == (0, 2816)


def test_captured_and_on_another_stream():
    s = _inputs(64, 2816, seed=8)
    want = B.block_norm(**s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = B.block_norm(**s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = B.block_norm(**s)
    torch.cuda.synchronize()
    other = _inputs(64, 2816, seed=9)
    for n in s:
        s[n].copy_(other[n])
    graph.replay()
    torch.cuda.synchronize()
    again = B.block_norm(**other)
    for i in range(2):
        assert torch.equal(got[i], want[i]) and torch.equal(held[i], again[i])


def test_refusals():
    s = _inputs(8, 64, seed=10)
    x, block, post, pre = s["x"], s["block"], s["post"], s["pre"]
    buf = torch.zeros(8 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    for kw, match in ((dict(x=x.float()), "bfloat16"), (dict(x=x[0]), "two dimensions"), (dict(x=x, post=post), "block"),
                      (dict(x=x, block=block[:4]), "block must be"), (dict(x=x, block=block, post=post[:8]), "post must hold"),
                      (dict(x=x, normed=block), "pre"), (dict(x=x.T.contiguous().T, pre=pre), "contiguous rows"),
                      (dict(x=x, block=block, post=post.cpu()), "post must be a contiguous tensor"),
                      (dict(x=x, pre=pre, normed=block[:, :8]), "normed must be"),
                      (dict(x=x[:, :12].contiguous(), scale=2.0), "multiple of 8")):
        with pytest.raises(ValueError, match=match):
            B.block_norm(**kw)
    for kw in (dict(x=x, pre=pre, eps=0.0), dict(x=x, pre=pre, eps=float("nan")), dict(x=x, pre=pre, scale=float("inf")),
               dict(x=x, block=block, out=s["gate"], gate=s["gate"]),
               dict(x=x, block=block, pre=pre, out=x, normed=x),
               dict(x=buf[:512].view(8, 64), block=block, out=buf[8:520].view(8, 64))):
        with pytest.raises(B.MoeFFNError):
            B.block_norm(**kw)
    with pytest.raises(B.MoeFFNError):  # too wide
        B.block_norm(torch.zeros(1, 16392, dtype=torch.bfloat16, device="cuda"), scale=2.0)


def test_places_past_32_bits():
    T, H = 800_000, 2816  # 2.25e9 elements
    rows = [0, 1, 762_599, 762_600, 799_999]  # (2^31 elements end in row 762600)
    small = _inputs(len(rows), H, seed=9, gate="one")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    n = torch.empty_like(x)
    x[rows] = small["x"]
    block = small["block"][:1].expand(T, H)
    B.block_norm(x, block, post=small["post"], gate=small["gate"][:1].expand(T, H), pre=small["pre"], out=x, normed=n)
    wy, wn, ty, tn = _wanted(**dict(small, block=small["block"][:1].expand(len(rows), H)))
    _check(x[rows], wy, ty)
    _check(n[rows], wn, tn)
    assert torch.equal(x[2], x[T - 2]) and torch.equal(n[2], n[T - 2])
