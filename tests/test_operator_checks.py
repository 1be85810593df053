"""Refusals of the norms, rotary positions, trees, kept paths, beams and their selection, and their structures' layout,
without a GPU: every call here fails its checks before it touches a pointer."""
import ctypes
import math
import os
import random
import subprocess
from fractions import Fraction

import pytest
import torch

from mixture_experts_ffn_router_gb300 import binding as B
from mixture_experts_ffn_router_gb300 import build as cuda_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AT = 1 << 20  # an address that is never looked at


@pytest.fixture(scope="module", autouse=True)
def built():
    cuda_build.build()


def test_layouts_and_limits_match_the_header(tmp_path):
    names = ("moe_ffn_norm", "moe_ffn_rotary_pair", "moe_ffn_rotary", "moe_ffn_beam")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_ffn.h"', "int main(void){"]
    for st in names:
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (st, st))
        for f, _ in getattr(B, st)._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (st, f, st, f))
    lines.append('printf("limits %d %d %d %d\\n", MOE_FFN_KV_TREE_NODES, MOE_FFN_BEAM_MAX, MOE_FFN_ROTARY_MAX_PAIRS, '
                 'MOE_FFN_ROTARY_MAX_AXES);return 0;}')
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
    assert got["limits"] == "%d %d %d %d" % (B.KV_TREE_NODES, B.BEAM_MAX, B.ROTARY_MAX_PAIRS, B.ROTARY_MAX_AXES)


# ------------------------------------------------------------------ norms

def _norm(**change):
    a = dict(x=AT, block=2 * AT, gate=None, post=3 * AT, pre=4 * AT, y=5 * AT, n=6 * AT, x_stride=64, block_stride=64,
             gate_stride=0, y_stride=64, n_stride=64, scale=1.0, eps=1e-6, tokens=4, hidden=64)
    a.update(change)
    return B.moe_ffn_norm(**a)


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(hidden=0), dict(hidden=12), dict(hidden=16392), dict(eps=0.0), dict(eps=-1e-6), dict(eps=math.nan),
    dict(eps=math.inf), dict(scale=math.nan), dict(scale=math.inf), dict(x=None), dict(y=None, n=None, pre=None), dict(pre=None),
    dict(n=None), dict(block=None), dict(block=None, post=None, gate=AT), dict(x_stride=-8), dict(block_stride=-8),
    dict(gate_stride=-8), dict(y_stride=56), dict(n_stride=0),
    dict(y=AT + 16), dict(y=AT, x_stride=72), dict(n=5 * AT), dict(n=5 * AT + 64 * 3), dict(y=3 * AT + 128), dict(n=4 * AT),
    dict(gate=5 * AT, gate_stride=64), dict(gate=6 * AT + 16), dict(y=AT + 64, y_stride=64, x_stride=128)])
def test_norm_refusals(change):
    assert B.moe_ffn_block_norm(_norm(**change), None) == B.MOE_FFN_EINVAL


@pytest.mark.parametrize("change", [dict(x=AT + 8), dict(block=AT + 2), dict(post=AT + 4), dict(pre=AT + 4), dict(y=AT + 8), dict(n=AT + 8),
                                    dict(gate=AT + 8), dict(x_stride=68), dict(y_stride=68), dict(gate=7 * AT, gate_stride=4)])
def test_norm_alignment(change):
    assert B.moe_ffn_block_norm(_norm(**change), None) == B.MOE_FFN_EALIGN


def test_norm_of_nothing():
    assert B.lib().moe_ffn_block_norm(None, None) == B.MOE_FFN_EINVAL
    assert B.moe_ffn_block_norm(_norm(tokens=0, x=None, y=None), None) == B.MOE_FFN_OK
    with pytest.raises(ValueError, match="CUDA"):
        B.block_norm(torch.zeros(2, 64, dtype=torch.bfloat16))


# ------------------------------------------------------------------ rotary positions

def test_turns_are_exact_fractions():
    """The table's turns against the frequency over 2 pi in exact arithmetic (pi to 60 digits): the quotient is a double's, good
    to 2^-51 of itself, then truncated to 2^-64."""
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
    freqs = [1.0, 1e4 ** -0.5, 1e-6, -0.3, 6.283185307179586, 12345.678, 0.0, 1e300, 5e-324, -1e-9]
    for (turn, axis), f, a in zip(B.moe_ffn_rotary_table(freqs, [i % 8 for i in range(10)]), freqs, range(10)):
        assert axis == a % 8
        if abs(f) > 1e20:
            continue  # no digit of the fraction is left
        exact = Fraction(f) / two_pi
        off = (Fraction(turn, 1 << 64) - exact) % 1
        off = min(off, 1 - off)
        assert off <= abs(exact) / (1 << 51) + Fraction(1, 1 << 64)


def _two_pi(bits):
    """2 pi to that many bits, by Machin's formula."""
    def arctan_of_inverse(n):
        total = power = (1 << (bits + 32)) // n
        k = sign = 1
        while power:
            power //= n * n
            k, sign = k + 2, -sign
            total += sign * (power // k)
        return total
    return Fraction(8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), 1 << (bits + 32))


def test_turns_are_rounded_once():
    """Every frequency's fraction of a turn is the exact quotient's, rounded to the nearest of 2^64."""
    two_pi = _two_pi(1400)
    rng = random.Random(5)
    freqs = [1.0, 1e4 ** -0.5, 1e-6, -0.3, 6.283185307179586, 12345.678, 1e6, 0.0, 1e300, -1.7976931348623157e308, 5e-324, -1e-9]
    freqs += [math.ldexp(f, e) for e in (-62, -61, -60, -59, -2, 2, 3, 64, 130) for f in (0.5, 0.75, 0.7853981633974482, 0.7853981633974483,
                                                                                         0.7853981633974484, 0.9999999999999999)]
    freqs += [math.ldexp(0.5 + rng.random() / 2, rng.randint(-70, 40)) for _ in range(200)]
    freqs += [math.ldexp(0.5 + rng.random() / 2, rng.randint(40, 1024)) for _ in range(100)]
    table = B.moe_ffn_rotary_table(freqs, [0] * len(freqs))
    for f, (turn, _) in zip(freqs, table):
        off = (Fraction(turn, 1 << 64) - Fraction(f) / two_pi) % 1
        assert min(off, 1 - off) <= Fraction(1, 1 << 65) * (1 + Fraction(1, 1 << 60)), f


def test_tables_are_checked():
    for freqs, axes in (([math.nan] * 4, [0] * 4), ([math.inf], [0]), ([1.0], [8]), ([1.0], [-1]), ([], []), ([1.0] * 513, [0] * 513)):
        with pytest.raises(B.MoeFFNError):
            B.moe_ffn_rotary_table(freqs, axes)
    with pytest.raises(ValueError):
        B.moe_ffn_rotary_table([1.0, 2.0], [0])
    for n in (0, 6, 516):
        with pytest.raises(ValueError, match="pairs"):
            B.Rotary([1.0] * n)


class _OnGpu:
    """In the place of a class's tensor argument: on a GPU as far as it says."""

    def __init__(self, *shape, dtype):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return AT


def test_a_table_stays_until_every_stream_is_done_with_it(monkeypatch):
    """The table belongs to the stream it was made on. Dropped while another one's call is queued, its memory must not
    go to new work before that; a call that is captured runs later, and says so nowhere."""
    raw, capturing, recorded = [1], [False], []
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: raw[0], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: raw[0])
    monkeypatch.setattr(B, "_launch", lambda call, device, *args: B.MOE_FFN_OK)
    monkeypatch.setattr(torch.Tensor, "to", lambda self, device: _Table())

    class _Table:
        def data_ptr(self):
            return AT

        def record_stream(self, stream):
            recorded.append(stream)

    r = B.Rotary([1.0] * 4)
    q, positions = _OnGpu(3, 2, 8, dtype=torch.bfloat16), _OnGpu(3, dtype=torch.int32)
    for raw[0], capturing[0] in ((1, False), (1, False), (2, False), (3, True), (3, True), (3, False), (1, False)):
        r.apply(q, None, positions, inplace=True)
    assert recorded == [1, 2, 3, 1]


def _rotary(rows=None, **change):
    a = dict(table=AT, positions=2 * AT, positions_stride=4, scale=1.0, pairs=32, axes=1, interleaved=0, inverse=0, tokens=4,
             head_dim=64, q_heads=2, k_heads=1)
    a.update(change)
    r = {n: B.moe_ffn_kv_rows(AT * (3 + i), 64 * (2 - i % 2), 64) for i, n in enumerate(("q", "k", "q_out", "k_out"))}
    for n, v in (rows or {}).items():
        r[n] = None if v is None else B.moe_ffn_kv_rows(*v)
    return B.moe_ffn_rotary_apply(B.moe_ffn_rotary(**a), r["q"], r["k"], r["q_out"], r["k_out"], None)


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(pairs=0), dict(pairs=6), dict(pairs=36), dict(pairs=516, head_dim=1032), dict(head_dim=60), dict(head_dim=1032),
    dict(axes=0), dict(axes=9), dict(q_heads=-1), dict(k_heads=1025), dict(scale=math.nan), dict(positions_stride=-1), dict(table=None),
    dict(positions=None), dict(rows=dict(q=None)), dict(rows=dict(k_out=None)), dict(rows=dict(q=(None, 128, 64))),
    dict(rows=dict(q=(3 * AT, -128, 64))),
    dict(rows=dict(q_out=(3 * AT + 128, 128, 64))),            # over the input, shifted
    dict(rows=dict(q_out=(3 * AT, 256, 64))),                  # the same place, other strides
    dict(rows=dict(q_out=(5 * AT, 64, 64))),                   # its own tokens overlap
    dict(rows=dict(q_out=(5 * AT, 128, 0))),
    dict(rows=dict(k_out=(5 * AT + 128, 64, 64))),             # over the other output
    dict(rows=dict(q_out=(4 * AT, 128, 64))),                  # over the other input
    dict(rows=dict(q_out=(AT, 128, 64))),                      # over the table
    dict(rows=dict(k_out=(2 * AT - 16, 64, 64)))])             # over the positions
def test_rotary_refusals(change):
    assert _rotary(**change) == B.MOE_FFN_EINVAL


@pytest.mark.parametrize("change", [dict(table=AT + 8), dict(positions=AT * 2 + 2), dict(rows=dict(q=(3 * AT + 8, 128, 64))),
                                    dict(rows=dict(k_out=(6 * AT, 68, 64))), dict(rows=dict(k=(4 * AT, 64, 4)))])
def test_rotary_alignment(change):
    assert _rotary(**change) == B.MOE_FFN_EALIGN


def test_rotary_of_nothing():
    assert _rotary(tokens=0, table=None, rows=dict(q=None)) == B.MOE_FFN_OK
    assert _rotary(q_heads=0, k_heads=0, table=None) == B.MOE_FFN_OK


# ------------------------------------------------------------------ selection

def _beam(workspace=10 * AT, nbytes=1 << 30, **change):
    a = dict(logits=AT, logits_stride=100, scores=20 * AT, finished=None, out_scores=30 * AT, out_beams=31 * AT, out_tokens=32 * AT,
             logits_fp32=0, end_token=0, users=2, beams=4, vocab=100, count=8)
    a.update(change)
    return B.moe_ffn_beam_select(B.moe_ffn_beam(**a), workspace, nbytes, None)


@pytest.mark.parametrize("change", [
    dict(users=-1), dict(users=4097), dict(beams=0), dict(beams=65), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(count=0),
    dict(count=65), dict(logits_stride=-1), dict(logits=None), dict(scores=None), dict(out_scores=None), dict(out_beams=None),
    dict(out_tokens=None), dict(workspace=None), dict(finished=AT * 40, end_token=-1), dict(finished=AT * 40, end_token=100),
    dict(out_beams=30 * AT + 60), dict(out_scores=20 * AT), dict(out_tokens=AT + 4), dict(out_tokens=10 * AT),
    dict(finished=32 * AT + 1), dict(workspace=AT)])
def test_selection_refusals(change):
    assert _beam(**change) == B.MOE_FFN_EINVAL


def test_selection_alignment_and_room():
    for change in (dict(logits=AT + 1), dict(logits=AT + 2, logits_fp32=1), dict(scores=20 * AT + 2), dict(out_beams=31 * AT + 1),
                   dict(workspace=10 * AT + 64)):
        assert _beam(**change) == B.MOE_FFN_EALIGN
    need = B.moe_ffn_beam_workspace_bytes(2, 4, 100, 8)
    assert need > 0 and _beam(nbytes=need - 1) == B.MOE_FFN_ETOOBIG
    assert _beam(users=0, logits=None) == B.MOE_FFN_OK
    assert B.lib().moe_ffn_beam_select(None, None, 0, None) == B.MOE_FFN_EINVAL
    for sizes in ((-1, 4, 100, 8), (4097, 1, 100, 8), (2, 65, 100, 8), (2, 4, 0, 8), (2, 4, 100, 0), (2, 4, 100, 65)):
        assert B.moe_ffn_beam_workspace_bytes(*sizes) == 0
        with pytest.raises(ValueError, match="invalid"):
            B.BeamSearch(*sizes)
    # The largest of each, and all of them together, have a size.
    assert B.moe_ffn_beam_workspace_bytes(4096, 64, 1 << 24, 64) > 4096 * 64 * 64 * 8


class _Streams:
    """In the place of torch's streams: what is done with the current one, in order."""

    def __init__(self, monkeypatch, capturing=False):
        self.done = []
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)

    def synchronize(self):
        self.done.append("synchronize")


@pytest.mark.parametrize("capturing", [False, True])
def test_a_search_waits_for_what_its_workspace_was(monkeypatch, capturing):
    """Work queued before on the stream that a search is made on may still write the memory that it gets; no call on
    another stream would wait for that."""
    streams = _Streams(monkeypatch, capturing)
    empty = torch.empty

    def allocate(*size, device=None, **kw):
        assert device == torch.device("cuda", 0)
        streams.done.append("allocate")
        return empty(*size, **kw)

    monkeypatch.setattr(torch, "empty", allocate)
    B.BeamSearch(2, 4, 100, 8)
    assert streams.done == (["allocate"] if capturing else ["allocate", "synchronize"])


# ------------------------------------------------------------------ the cache's calls

def test_calls_without_a_handle():
    L = B.lib()
    c, b, r = B.moe_ffn_kv_cache(), B.moe_ffn_kv_batch(), B.moe_ffn_kv_rows()
    assert L.moe_ffn_kv_tree(None, b, None, None, None, None) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_tree_attention(None, c, b, None, r, 1.0, 0, 0, None, None, None) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_tree_attention(None, c, None, None, r, 1.0, 0, 0, None, None, None) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_keep(None, ctypes.byref(c), 1, b, None, 0, 0, None, None, None) == B.MOE_FFN_EINVAL
    assert L.moe_ffn_kv_reorder(None, ctypes.byref(c), 1, None, 0, 0, None, None, 0, 1, None) == B.MOE_FFN_EINVAL


def _stub():
    """A PagedKV without a device: what its argument checks read."""
    kv = B.PagedKV.__new__(B.PagedKV)
    kv.ctx, kv.fmt, kv.device = 0, "bf16", torch.device("cuda", 0)
    kv.q_heads, kv.kv_heads, kv.head_dim, kv.shape = 16, 8, 256, (10, 8, 64, 256)
    kv.dtype, kv._kind = torch.bfloat16, None
    return kv


def test_masks_stay_until_every_stream_is_done_with_them(monkeypatch):
    """A tree's masks belong to the stream that made them; its attention may be queued on another one when it is dropped."""
    raw, capturing, recorded = [1], [False], []

    class Masks(_OnGpu):
        def record_stream(self, stream):
            recorded.append(stream)

    kv = _stub()
    kv._handle, kv.default_scale = None, 1.0
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *size, dtype=None, device=None: empty(*size, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: raw[0])
    monkeypatch.setattr(kv, "_rows", lambda *a: None, raising=False)
    monkeypatch.setattr(kv, "_begin", lambda cache, batch: (None, raw[0]), raising=False)
    monkeypatch.setattr(B, "moe_ffn_kv_tree_attention", lambda *a: B.MOE_FFN_OK)
    batch = B.KVBatch.__new__(B.KVBatch)
    batch.of = lambda n: None
    tree = B.KVTree(Masks(4, 8, dtype=torch.int32), None, 1)
    q = torch.zeros(4, 16, 256, dtype=torch.bfloat16)
    for raw[0], capturing[0] in ((1, False), (2, False), (3, True), (3, False), (1, False)):
        kv.tree_attention(None, batch, tree, q)
    assert recorded == [2, 3]


def test_arguments_of_the_cache_are_checked():
    kv = _stub()
    ids = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    batch = B.KVBatch.__new__(B.KVBatch)
    batch.tensors, batch.device = (ids(3), ids(2), ids(2, 4)), kv.device
    for call, match in ((lambda: kv.tree(batch, ids(5, 1)), "one dimension"), (lambda: kv.tree(batch, ids(5).long()), "int32"),
                        (lambda: kv.tree(batch, ids(5)), "contiguous tensor on cuda"),
                        (lambda: kv.keep([], batch, ids(2), ids(2)), "two dimensions"),
                        (lambda: kv.keep([], batch, ids(3, 4), ids(2)), "nodes must be"),
                        (lambda: kv.reorder([], ids(4, 2), ids(2), ids(4)), "two dimensions"),
                        (lambda: kv.reorder([], ids(4, 2), ids(2), ids(2, 2).float()), "parents must be"),
                        (lambda: kv.tree_attention(None, batch, B.KVTree(ids(5, 8), ids(5)), torch.zeros(4, 16, 256)), "tokens")):
        with pytest.raises(ValueError, match=match):
            call()
