"""The paged cache's refusals, and its structures' layout, without a GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

from mixture_experts_ffn_router_gb300 import binding as B
from mixture_experts_ffn_router_gb300 import build as cuda_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = dict(q_heads=16, kv_heads=8, head_dim=256, page_size=64, n_pages=10, fmt="bf16", max_tokens=64, max_seqs=4)


@pytest.fixture(scope="module", autouse=True)
def built():
    cuda_build.build()


def test_struct_layouts_match_the_header(tmp_path):
    names = ("moe_ffn_kv_config", "moe_ffn_kv_cache", "moe_ffn_kv_batch", "moe_ffn_kv_rows")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_ffn.h"', "int main(void){"]
    for st in names:
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (st, st))
        for f, _ in getattr(B, st)._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (st, f, st, f))
    lines.append('printf("formats %d %d\\n", MOE_FFN_KV_BF16, MOE_FFN_KV_E4M3);return 0;}')
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = dict(l.split(" ", 1) for l in out.strip().split("\n"))
    for st in names:
        cls = getattr(B, st)
        assert int(got[st]) == ctypes.sizeof(cls), st
        for f, _ in cls._fields_:
            assert int(got["%s.%s" % (st, f)]) == getattr(cls, f).offset, (st, f)
    assert got["formats"] == "%d %d" % (B.KV_FORMATS["bf16"], B.KV_FORMATS["e4m3"])


def test_workspace_of_a_good_configuration():
    assert B.moe_ffn_kv_workspace_bytes(B.make_kv_config(**GOOD)) >= 256


@pytest.mark.parametrize("change", [
    dict(q_heads=0), dict(kv_heads=0), dict(q_heads=12), dict(q_heads=8 * 65), dict(head_dim=64), dict(head_dim=192),
    dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(n_pages=0), dict(n_pages=1 << 22),
    dict(fmt="int4"), dict(max_tokens=0), dict(max_tokens=(1 << 24) + 1), dict(max_seqs=0), dict(max_seqs=65537)])
def test_bad_configurations_have_no_workspace(change):
    assert B.moe_ffn_kv_workspace_bytes(B.make_kv_config(**{**GOOD, **change})) == 0


def test_calls_without_a_handle():
    L = B.lib()
    c, b, r = B.moe_ffn_kv_cache(), B.moe_ffn_kv_batch(), B.moe_ffn_kv_rows()
    assert L.moe_ffn_kv_write(None, c, b, r, r, None) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_read(None, c, b, None, None, None) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_attention(None, c, b, r, 1.0, 0, 0, None, None, None) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_device_status(None, None, None) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_init(None, None, None, 0, 0) == B.MOE_FFN_EINVAL
    h = ctypes.c_void_p(4096)
    cfg = B.make_kv_config(**GOOD)
    assert L.moe_ffn_kv_init(ctypes.byref(h), ctypes.byref(cfg), None, 1 << 30, 0) == B.MOE_FFN_EINVAL
    assert not h.value
    assert L.moe_ffn_kv_init(ctypes.byref(h), ctypes.byref(cfg), ctypes.c_void_p(4096 + 16), 1 << 30,
                             0) == B.MOE_FFN_EALIGN
    assert L.moe_ffn_kv_init(ctypes.byref(h), ctypes.byref(cfg), ctypes.c_void_p(4096), 16, 0) == B.MOE_FFN_ETOOBIG
    L.moe_ffn_kv_destroy(None)


def test_format_and_configuration_are_named():
    with pytest.raises(ValueError, match="fmt"):
        B.PagedKV(16, 8, 256, 64, 10, "fp8")
    with pytest.raises(ValueError, match="invalid configuration"):
        B.PagedKV(16, 8, 100, 64, 10)


def _stub(fmt="bf16"):
    """A PagedKV without a device: what its argument checks read."""
    kv = B.PagedKV.__new__(B.PagedKV)
    kv.ctx, kv.fmt, kv.device = 0, fmt, torch.device("cuda", 0)
    kv.q_heads, kv.kv_heads, kv.head_dim, kv.shape = 16, 8, 256, (10, 8, 64, 256)
    kv.dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    return kv


@pytest.mark.parametrize("shape,dtype,match", [
    ((3, 16, 256), torch.float32, "bfloat16"), ((3, 8, 256), torch.bfloat16, "shape"),
    ((3, 16, 128), torch.bfloat16, "shape"), ((3, 4096), torch.bfloat16, "shape"),
    ((3, 16, 256), torch.bfloat16, "must be on")])
def test_queries_are_checked(shape, dtype, match):
    with pytest.raises(ValueError, match=match):
        _stub()._rows("q", torch.empty(shape, dtype=dtype, device="meta"), 16)


@pytest.mark.parametrize("fmt,change,match", [
    ("bf16", dict(k=None), "required"), ("bf16", dict(v_scale="scale"), "no scales"),
    ("bf16", dict(v=torch.float8_e4m3fn), "v must be"), ("e4m3", dict(k_scale=None), "k_scale is required"),
    ("e4m3", dict(v_scale=torch.float64), "v_scale must be"), ("e4m3", dict(k="short"), "k must be"),
    ("e4m3", dict(), "CUDA tensor")])
def test_caches_are_checked(fmt, change, match):
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    given = {n: torch.empty((10, 8, 64, 256), dtype=dtype, device="meta") for n in ("k", "v")}
    if fmt == "e4m3":
        given.update({n: torch.empty((10, 8, 64), device="meta") for n in ("k_scale", "v_scale")})
    for n, what in change.items():
        if isinstance(what, torch.dtype):
            given[n] = torch.empty(given[n].shape, dtype=what, device="meta")
        elif what == "short":
            given[n] = given[n][:, :, :32]
        elif what == "scale":
            given[n] = torch.empty((10, 8, 64), device="meta")
        else:
            given[n] = None
    with pytest.raises(ValueError, match=match):
        _stub(fmt).cache(**given)


def _meta_cache(shape, dtype, scales, kind=None):
    c = B.KVCache(*(torch.empty(shape, dtype=dtype, device="meta") for _ in range(2)),
                  *(torch.empty(shape[:3], device="meta") for _ in range(2 if scales else 0)))
    c.kind = kind
    return c


@pytest.mark.parametrize("shape,dtype,scales", [
    ((10, 2, 64, 512), torch.bfloat16, False), ((9, 8, 64, 256), torch.bfloat16, False),
    ((10, 8, 32, 256), torch.bfloat16, False), ((10, 8, 64, 256), torch.float8_e4m3fn, True),
    ((10, 8, 64, 256), torch.float16, False)])
def test_caches_of_another_handle_are_checked(shape, dtype, scales):
    """A cache made for another shape, format or device is refused before anything is launched."""
    kv = _stub()
    kv._kind = ((10, 8, 64, 256), torch.bfloat16, kv.device)
    for kind in (None, (shape, dtype, kv.device)):
        c = _meta_cache(shape, dtype, scales, kind)
        with pytest.raises(ValueError, match="must be|has no scales"):
            kv._begin(c, None)
    other = _meta_cache((10, 8, 64, 256), torch.bfloat16, False, ((10, 8, 64, 256), torch.bfloat16, torch.device("cuda", 1)))
    with pytest.raises(ValueError, match="CUDA tensor"):
        kv._begin(other, None)


class _OnDevice:
    """What KVBatch's checks read of a CUDA tensor."""
    is_cuda, dtype, device = True, torch.int32, torch.device("cuda", 0)

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return (self.shape[1], 1)[i] if len(self.shape) == 2 else 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def test_a_batch_given_to_one_call_is_not_changed_by_the_next():
    """Threads with a handle each may share a batch, for tensors of different token counts."""
    batch = B.KVBatch(_OnDevice(5), _OnDevice(4), _OnDevice(4, 2), max_new=3)
    given = [batch.of(n) for n in (3, 5, 5, 3)]
    structs = [ctypes.cast(g, ctypes.POINTER(B.moe_ffn_kv_batch)).contents for g in given]
    assert [s.n_tokens for s in structs] == [3, 5, 5, 3]
    assert all((s.n_seqs, s.pages_cols, s.pages_stride, s.max_new, s.cu_q) == (4, 2, 2, 3, 4096) for s in structs)


def test_operators_go_through_the_c_entry_points(monkeypatch):
    seen = []
    for name in ("moe_ffn_kv_write", "moe_ffn_kv_read", "moe_ffn_kv_attention"):
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append((name, a[0], a[2], a[-1])) or B.MOE_FFN_OK)
    kv = _stub()
    kv._handle, kv.default_scale = 11, 0.1
    kv._begin = lambda cache, batch: ("cache", 7)
    kv._rows = lambda what, t, heads: what
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: torch.zeros(1))
    batch = type("Batch", (), {"of": lambda self, n: ("batch", n)})()
    x = torch.zeros(3, 1, 1)
    kv.write(None, batch, x, x)
    kv.read(None, batch, 2)
    kv.attention(None, batch, x)
    assert seen == [("moe_ffn_kv_write", 11, ("batch", 3), 7), ("moe_ffn_kv_read", 11, ("batch", 2), 7),
                    ("moe_ffn_kv_attention", 11, ("batch", 3), 7)]


@pytest.mark.parametrize("given,passed", [(0, 0), (1024, 1024), (-1, -1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                          (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63 - 1, 2 ** 31 - 1), (-2 ** 32, -1)])
def test_windows_and_sinks_of_any_size_keep_their_meaning(monkeypatch, given, passed):
    """A C int would keep their lowest 32 bits."""
    seen = []
    monkeypatch.setattr(B, "moe_ffn_kv_attention", lambda *a: seen.append(a[5:7]) or B.MOE_FFN_OK)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: torch.zeros(1))
    kv = _stub()
    kv._handle, kv.default_scale = 11, 0.1
    kv._begin = lambda cache, batch: ("cache", 7)
    kv._rows = lambda what, t, heads: what
    batch = type("Batch", (), {"of": lambda self, n: ("batch", n)})()
    kv.attention(None, batch, torch.zeros(3, 1, 1), window=given, sinks=given)
    assert seen == [(passed, passed)]


def test_calls_after_close_are_refused(monkeypatch):
    monkeypatch.setattr(B, "moe_ffn_kv_destroy", lambda kv: None)
    kv = _stub()
    kv.ctx, kv._handle, kv._lib, kv.default_scale = 4096, ctypes.c_void_p(4096), B.lib(), 0.1
    kv._begin = lambda cache, batch: (B.moe_ffn_kv_cache(), 0)
    kv._rows = lambda what, t, heads: B.moe_ffn_kv_rows()
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: torch.zeros(1))

    class Batch:
        def of(self, n):
            return B.moe_ffn_kv_batch()

    kv.close()
    assert not kv.ctx and not kv._handle  # before any call: the C side cannot tell a handle that is gone
    x = torch.zeros(1, 1, 1)
    for call in (lambda: kv.write(None, Batch(), x, x), lambda: kv.read(None, Batch(), 1),
                 lambda: kv.attention(None, Batch(), x)):
        with pytest.raises(B.MoeFFNError) as e:
            call()
        assert e.value.status == B.MOE_FFN_EINVAL
    kv.close()


def test_the_workspace_is_held_for_each_stream_it_is_used_on(monkeypatch):
    """The allocator must not hand the workspace on while another stream than the one it was made on uses it."""
    class Stream:
        def __init__(self, raw):
            self.raw, self.waited = raw, []

        def wait_stream(self, other):
            self.waited.append(other)

    now = {"stream": None, "capturing": False}
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: now["stream"].raw, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    kv = _stub()
    kv._kind = (kv.shape, kv.dtype, kv.device)
    kv._last = kv._last_raw = None
    held = []
    kv.workspace = type("Workspace", (), {"record_stream": lambda self, stream: held.append(stream)})()
    cache = _meta_cache(kv.shape, kv.dtype, False, kv._kind)
    batch = type("Batch", (), {"device": kv.device})()
    a, b = Stream(7), Stream(9)
    for stream, capturing in ((a, False), (a, False), (b, False), (b, True), (a, True), (a, False)):
        now.update(stream=stream, capturing=capturing)
        assert kv._begin(cache, batch)[1] == stream.raw
    assert held == [a, b, a]
    assert b.waited == [a] and a.waited == [b]


@pytest.mark.parametrize("cu,kv,pages,new,match", [
    ((4,), (4,), (4, 2), 1, "sequences"), ((5,), (4,), (3, 2), 1, "sequences"), ((5,), (4, 1), (4, 2), 1, "dimension"),
    ((5,), (4,), (4,), 1, "dimension"), ((5,), (4,), (4, 2), -1, "max_new"), ((5,), (4,), (4, 2), 1, "CUDA tensor")])
def test_batches_are_checked(cu, kv, pages, new, match):
    t = [torch.empty(s, dtype=torch.int32, device="meta") for s in (cu, kv, pages)]
    with pytest.raises(ValueError, match=match):
        B.KVBatch(*t, max_new=new)
    if match == "CUDA tensor":
        with pytest.raises(ValueError, match="int32"):
            B.KVBatch(t[0].long(), *t[1:], max_new=new)
