"""ctypes binding of the C ABI in include/moe_ffn.h (argument marshalling only).

The functions keep the C names and take plain integers for device pointers and streams. ``MoeFFN``
is a small convenience wrapper that takes torch tensors (torch supplies device memory and the
stream; every step of the block runs in the library's kernels). Loading fails loudly when the
library has not been built: there is no fallback.
"""
import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_ffn.so")

MOE_FFN_OK = 0
MOE_FFN_EINVAL = -1
MOE_FFN_EALIGN = -2
MOE_FFN_ETOOBIG = -3
MOE_FFN_EARCH = -4
MOE_FFN_ECUDA = -5
MOE_FFN_EDEVICE = -6
MOE_FFN_MOE_ONLY = 0
MOE_FFN_FULL_LAYER = 1
HIDDEN, N_EXPERTS, TOP_K, MOE_INTER, DENSE_INTER = 2816, 128, 8, 704, 2112
# Bits of the device status word (MOE_FFN_STATUS_* in include/moe_ffn.h).
STATUS_BITS = {"WAIT_FULL": 0x1, "WAIT_EMPTY": 0x2, "WAIT_ACC_FULL": 0x4, "WAIT_ACC_EMPTY": 0x8,
               "BAD_INDEX": 0x10, "BAD_SCHEDULE": 0x20, "DRAIN": 0x40, "WAIT_ITEM": 0x80,
               "WAIT_COPY": 0x100}


def decode_status(word: int) -> list:
    """Names of the bits set in a device status word, lowest first; unknown bits as hex."""
    names = [n for n, b in sorted(STATUS_BITS.items(), key=lambda kv: kv[1]) if word & b]
    rest = word & ~sum(STATUS_BITS.values())
    return names + (["0x%x" % rest] if rest else [])


KERNEL_NAMES = ("router_prep", "router_logits", "route_topk", "route_scatter", "gate_up_gemm", "down_gemm", "combine")
# Forwards of at most this many tokens run the whole routing front end (router sums, top-k,
# counting sort) as one kernel in slot 1; slots 0, 2 and 3 then launch nothing.
ROUTE_SMALL_T = 64


def slot_name(slot: int, T: int) -> str:
    """Name of the kernel a forward of T tokens launches in kernel slot `slot`."""
    if slot == 1 and T <= ROUTE_SMALL_T:
        return "route_small"
    return KERNEL_NAMES[slot]

_vp = ctypes.c_void_p


class moe_ffn_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int),
                ("moe_inter", ctypes.c_int), ("dense_inter", ctypes.c_int), ("mode", ctypes.c_int),
                ("max_tokens", ctypes.c_int), ("eps", ctypes.c_float), ("router_scale", ctypes.c_float)]


WEIGHT_FIELDS = ("router_w", "router_norm_w", "per_expert_scale", "gate_up", "down", "dense_gate", "dense_up",
                 "dense_down", "pre_ff_ln", "pre_ff_ln_2", "post_ff_ln_1", "post_ff_ln_2", "post_ff_ln")


INT8_FIELDS = ("gate_up_q", "gate_up_scale", "down_q", "down_scale")
F4_FIELDS = ("gate_up_f4", "gate_up_f4s", "down_f4", "down_f4s")


class moe_ffn_weights(ctypes.Structure):
    _fields_ = ([(f, _vp) for f in WEIGHT_FIELDS] + [("layer_scalar", ctypes.c_float)] + [(f, _vp) for f in INT8_FIELDS]
                + [(f, _vp) for f in F4_FIELDS])


VIEW_FIELDS = ("logits", "topk_idx", "topk_w", "gap", "counts", "offsets", "perm", "w_sorted", "slot_pos", "n1",
               "n2", "h", "h_dense", "y", "d")


class moe_ffn_views(ctypes.Structure):
    _fields_ = [(f, _vp) for f in VIEW_FIELDS] + [("T", ctypes.c_int)]


KV_FORMATS = {"bf16": 0, "e4m3": 1}  # MOE_FFN_KV_BF16, MOE_FFN_KV_E4M3


class moe_ffn_kv_config(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("q_heads", "kv_heads", "head_dim", "page_size", "n_pages", "format",
                                            "max_tokens", "max_seqs")]


class moe_ffn_kv_cache(ctypes.Structure):
    _fields_ = [(f, _vp) for f in ("k", "v", "k_scale", "v_scale")]


class moe_ffn_kv_batch(ctypes.Structure):
    _fields_ = ([(f, _vp) for f in ("cu_q", "kv_len", "pages")] + [("pages_stride", ctypes.c_longlong)]
                + [(f, ctypes.c_int) for f in ("pages_cols", "n_seqs", "n_tokens", "max_new")])


class moe_ffn_kv_rows(ctypes.Structure):
    _fields_ = [("ptr", _vp), ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


KV_TREE_NODES, BEAM_MAX, ROTARY_MAX_PAIRS, ROTARY_MAX_AXES = 256, 64, 512, 8  # as include/moe_ffn.h has them


class moe_ffn_norm(ctypes.Structure):
    _fields_ = ([(f, _vp) for f in ("x", "block", "gate", "post", "pre", "y", "n")]
                + [(f, ctypes.c_longlong) for f in ("x_stride", "block_stride", "gate_stride", "y_stride", "n_stride")]
                + [("scale", ctypes.c_float), ("eps", ctypes.c_float), ("tokens", ctypes.c_int), ("hidden", ctypes.c_int)])


class moe_ffn_rotary_pair(ctypes.Structure):
    _fields_ = [("turn", ctypes.c_uint64), ("axis", ctypes.c_uint64)]


class moe_ffn_rotary(ctypes.Structure):
    _fields_ = ([("table", _vp), ("positions", _vp), ("positions_stride", ctypes.c_longlong), ("scale", ctypes.c_float)]
                + [(f, ctypes.c_int) for f in ("pairs", "axes", "interleaved", "inverse", "tokens", "head_dim", "q_heads",
                                               "k_heads")])


class moe_ffn_beam(ctypes.Structure):
    _fields_ = ([("logits", _vp), ("logits_stride", ctypes.c_longlong)]
                + [(f, _vp) for f in ("scores", "finished", "out_scores", "out_beams", "out_tokens")]
                + [(f, ctypes.c_int) for f in ("logits_fp32", "end_token", "users", "beams", "vocab", "count")])


# Some calls' structures are packed into bytes: a ctypes structure of a dozen fields takes longer than the call.
_PACK_NORM = struct.Struct("@7P5q2f2i").pack
_PACK_ROTARY = struct.Struct("@2Pqf8i4x").pack
_PACK_ROWS = struct.Struct("@Pqq").pack
_PACK_BEAM = struct.Struct("@Pq5P6i").pack


def _by_ref(s):
    """A structure, or one that is packed or absent already, as an argument."""
    return ctypes.byref(s) if isinstance(s, ctypes.Structure) else s


_LIB = None


def lib():
    """The loaded CUDA library. Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe_ffn.so is not built (run __graft_entry__.build() or "
                               "python mixture_experts_ffn_router_gb300/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_ffn_workspace_bytes.restype = ctypes.c_size_t
        L.moe_ffn_workspace_bytes.argtypes = [ctypes.POINTER(moe_ffn_config)]
        L.moe_ffn_init.restype = ctypes.c_int
        L.moe_ffn_init.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(moe_ffn_config), _vp, ctypes.c_size_t,
                                   ctypes.c_int]
        L.moe_ffn_forward.restype = ctypes.c_int
        L.moe_ffn_forward.argtypes = [_vp, _vp, ctypes.c_int, ctypes.POINTER(moe_ffn_weights), _vp, _vp]
        L.moe_ffn_forward_shard.restype = ctypes.c_int
        L.moe_ffn_forward_shard.argtypes = [_vp, _vp, ctypes.c_int, ctypes.POINTER(moe_ffn_weights), ctypes.c_int,
                                            ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]
        L.moe_ffn_finish_shards.restype = ctypes.c_int
        L.moe_ffn_finish_shards.argtypes = [_vp, _vp, ctypes.c_int, ctypes.POINTER(moe_ffn_weights), _vp, _vp, _vp,
                                            _vp]
        L.moe_ffn_workspace_view.restype = ctypes.c_int
        L.moe_ffn_workspace_view.argtypes = [_vp, ctypes.POINTER(moe_ffn_views)]
        L.moe_ffn_device_status.restype = ctypes.c_int
        L.moe_ffn_device_status.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_uint32)]
        L.moe_ffn_set_kernel_events.restype = ctypes.c_int
        L.moe_ffn_set_kernel_events.argtypes = [_vp, ctypes.c_int, _vp, _vp]
        L.moe_ffn_kernels_per_forward.restype = ctypes.c_int
        L.moe_ffn_kernels_per_forward.argtypes = [_vp, ctypes.c_int]
        L.moe_ffn_kernel_slots.restype = ctypes.c_int
        L.moe_ffn_kernel_slots.argtypes = [_vp, ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.c_int]
        L.moe_ffn_router_logits_noalloc.restype = ctypes.c_int
        L.moe_ffn_router_logits_noalloc.argtypes = [_vp, ctypes.c_int, _vp, _vp, ctypes.c_float, ctypes.c_float,
                                                     _vp, _vp]
        L.moe_ffn_selftest_wait_expiry.restype = ctypes.c_int
        L.moe_ffn_selftest_wait_expiry.argtypes = [_vp, _vp, _vp]
        L.moe_ffn_status_string.restype = ctypes.c_char_p
        L.moe_ffn_status_string.argtypes = [ctypes.c_int]
        L.moe_ffn_quantize_int8.restype = ctypes.c_int
        L.moe_ffn_quantize_int8.argtypes = [_vp, ctypes.c_longlong, ctypes.c_int, _vp, _vp, _vp]
        L.moe_ffn_quantize_mxfp4.restype = ctypes.c_int
        L.moe_ffn_quantize_mxfp4.argtypes = [_vp, ctypes.c_longlong, ctypes.c_int, _vp, _vp, _vp]
        cfg_p, cache_p, batch_p, rows_p = (ctypes.POINTER(t) for t in (moe_ffn_kv_config, moe_ffn_kv_cache,
                                                                       moe_ffn_kv_batch, moe_ffn_kv_rows))
        L.moe_ffn_kv_workspace_bytes.restype = ctypes.c_size_t
        L.moe_ffn_kv_workspace_bytes.argtypes = [cfg_p]
        L.moe_ffn_kv_init.restype = ctypes.c_int
        L.moe_ffn_kv_init.argtypes = [ctypes.POINTER(_vp), cfg_p, _vp, ctypes.c_size_t, ctypes.c_int]
        L.moe_ffn_kv_write.restype = ctypes.c_int
        L.moe_ffn_kv_write.argtypes = [_vp, cache_p, batch_p, rows_p, rows_p, _vp]
        L.moe_ffn_kv_read.restype = ctypes.c_int
        L.moe_ffn_kv_read.argtypes = [_vp, cache_p, batch_p, _vp, _vp, _vp]
        L.moe_ffn_kv_attention.restype = ctypes.c_int
        L.moe_ffn_kv_attention.argtypes = [_vp, cache_p, batch_p, rows_p, ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                           _vp, _vp, _vp]
        L.moe_ffn_kv_device_status.restype = ctypes.c_int
        L.moe_ffn_kv_device_status.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_uint32)]
        L.moe_ffn_kv_destroy.restype = None
        L.moe_ffn_kv_destroy.argtypes = [_vp]
        L.moe_ffn_kv_tree.restype = ctypes.c_int
        L.moe_ffn_kv_tree.argtypes = [_vp, batch_p, _vp, _vp, _vp, _vp]
        L.moe_ffn_kv_tree_attention.restype = ctypes.c_int
        L.moe_ffn_kv_tree_attention.argtypes = [_vp, cache_p, batch_p, _vp, rows_p, ctypes.c_float, ctypes.c_int,
                                                ctypes.c_int, _vp, _vp, _vp]
        L.moe_ffn_kv_keep.restype = ctypes.c_int
        L.moe_ffn_kv_keep.argtypes = [_vp, _vp, ctypes.c_int, batch_p, _vp, ctypes.c_longlong, ctypes.c_int, _vp, _vp,
                                      _vp]
        L.moe_ffn_kv_reorder.restype = ctypes.c_int
        L.moe_ffn_kv_reorder.argtypes = [_vp, _vp, ctypes.c_int, _vp, ctypes.c_longlong, ctypes.c_int, _vp, _vp,
                                         ctypes.c_int, ctypes.c_int, _vp]
        L.moe_ffn_block_norm.restype = ctypes.c_int
        L.moe_ffn_block_norm.argtypes = [_vp, _vp]
        L.moe_ffn_rotary_table.restype = ctypes.c_int
        L.moe_ffn_rotary_table.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int), ctypes.c_int,
                                           ctypes.POINTER(moe_ffn_rotary_pair)]
        L.moe_ffn_rotary_apply.restype = ctypes.c_int
        L.moe_ffn_rotary_apply.argtypes = [_vp] * 6
        L.moe_ffn_beam_workspace_bytes.restype = ctypes.c_size_t
        L.moe_ffn_beam_workspace_bytes.argtypes = [ctypes.c_int] * 4
        L.moe_ffn_beam_select.restype = ctypes.c_int
        L.moe_ffn_beam_select.argtypes = [_vp, _vp, ctypes.c_size_t, _vp]
        L.moe_ffn_destroy.restype = None
        L.moe_ffn_destroy.argtypes = [_vp]
        _LIB = L
    return _LIB


class MoeFFNError(RuntimeError):
    def __init__(self, call, status):
        self.status = status
        super().__init__("%s: %s (%d)" % (call, moe_ffn_status_string(status), status))


def _check(call, status):
    if status != MOE_FFN_OK:
        raise MoeFFNError(call, status)
    return status


# ------------------------------------------------------------------ the C entry points

def moe_ffn_status_string(status: int) -> str:
    return lib().moe_ffn_status_string(int(status)).decode()


def make_config(mode: int, max_tokens: int, eps: float = 1e-6, router_scale: float = HIDDEN ** -0.5) -> moe_ffn_config:
    return moe_ffn_config(HIDDEN, N_EXPERTS, TOP_K, MOE_INTER, DENSE_INTER, int(mode), int(max_tokens),
                          float(eps), float(router_scale))


def moe_ffn_workspace_bytes(cfg: moe_ffn_config) -> int:
    return lib().moe_ffn_workspace_bytes(ctypes.byref(cfg))


def moe_ffn_init(cfg: moe_ffn_config, workspace: int, workspace_bytes: int, device: int) -> int:
    """Returns the context handle (an int)."""
    h = _vp()
    _check("moe_ffn_init", lib().moe_ffn_init(ctypes.byref(h), ctypes.byref(cfg), _vp(workspace),
                                               workspace_bytes, int(device)))
    return h.value


def moe_ffn_forward(ctx: int, x: int, T: int, weights: moe_ffn_weights, out: int, stream: int) -> int:
    return lib().moe_ffn_forward(_vp(ctx), _vp(x), int(T), ctypes.byref(weights), _vp(out), _vp(stream))


def moe_ffn_forward_shard(ctx: int, x: int, T: int, weights: moe_ffn_weights, expert_begin: int, expert_end: int,
                          with_dense: bool, moe_partial: int, dense_out: int, stream: int) -> int:
    return lib().moe_ffn_forward_shard(_vp(ctx), _vp(x), int(T), ctypes.byref(weights), int(expert_begin),
                                       int(expert_end), 1 if with_dense else 0, _vp(moe_partial), _vp(dense_out),
                                       _vp(stream))


def moe_ffn_finish_shards(ctx: int, x: int, T: int, weights: moe_ffn_weights, moe_sum: int, dense: int, out: int,
                          stream: int) -> int:
    return lib().moe_ffn_finish_shards(_vp(ctx), _vp(x), int(T), ctypes.byref(weights), _vp(moe_sum), _vp(dense),
                                       _vp(out), _vp(stream))


def expert_range(rank: int, world: int, n_experts: int = N_EXPERTS):
    """The contiguous experts [begin, end) that rank `rank` of `world` owns (equal shares, the first
    n_experts % world ranks one more)."""
    base, extra = divmod(n_experts, world)
    begin = rank * base + min(rank, extra)
    return begin, begin + base + (1 if rank < extra else 0)


def moe_ffn_workspace_view(ctx: int) -> moe_ffn_views:
    v = moe_ffn_views()
    _check("moe_ffn_workspace_view", lib().moe_ffn_workspace_view(_vp(ctx), ctypes.byref(v)))
    return v


def moe_ffn_device_status(ctx: int, stream: int):
    w = ctypes.c_uint32(0)
    rc = lib().moe_ffn_device_status(_vp(ctx), _vp(stream), ctypes.byref(w))
    return rc, w.value


def moe_ffn_set_kernel_events(ctx: int, kernel: int, start: int, stop: int) -> int:
    return lib().moe_ffn_set_kernel_events(_vp(ctx), int(kernel), _vp(start), _vp(stop))


def moe_ffn_kernels_per_forward(ctx: int, T: int) -> int:
    return lib().moe_ffn_kernels_per_forward(_vp(ctx), int(T))


def moe_ffn_kernel_slots(ctx: int, T: int) -> list:
    """The kernel slots a forward of T tokens launches, in launch order."""
    buf = (ctypes.c_int * len(KERNEL_NAMES))()
    n = lib().moe_ffn_kernel_slots(_vp(ctx), int(T), buf, len(KERNEL_NAMES))
    if n < 0:
        raise MoeFFNError("moe_ffn_kernel_slots", n)
    return list(buf[:n])


def moe_ffn_router_logits_noalloc(x: int, T: int, router_w: int, router_norm_w: int, router_scale: float,
                                  eps: float, logits: int, stream: int) -> int:
    """Router logits [T, 128] fp32 without any device allocation by the library (for callers that
    cannot allocate); its scratch is a fixed array shared by all calls, see include/moe_ffn.h."""
    return lib().moe_ffn_router_logits_noalloc(_vp(x), int(T), _vp(router_w), _vp(router_norm_w),
                                               float(router_scale), float(eps), _vp(logits), _vp(stream))


def moe_ffn_selftest_wait_expiry(status_word: int, record: int, stream: int) -> int:
    return lib().moe_ffn_selftest_wait_expiry(_vp(status_word), _vp(record), _vp(stream))


def moe_ffn_quantize_int8(w: int, rows: int, cols: int, q: int, scale: int, stream: int) -> int:
    return lib().moe_ffn_quantize_int8(_vp(w), int(rows), int(cols), _vp(q), _vp(scale), _vp(stream))


def quantize_experts_int8(w: dict) -> dict:
    """Adds the int8 form of the experts (gate_up_q/scale, down_q/scale) to a dict of CUDA weight
    tensors, made on the device by moe_ffn_quantize_int8."""
    import torch
    out = dict(w)
    s = torch.cuda.current_stream().cuda_stream
    for name, rows, cols in (("gate_up", N_EXPERTS * 2 * MOE_INTER, HIDDEN), ("down", N_EXPERTS * HIDDEN, MOE_INTER)):
        src = w[name]
        q = torch.empty((rows, cols), dtype=torch.int8, device=src.device)
        sc = torch.empty(rows, dtype=torch.float32, device=src.device)
        _check("moe_ffn_quantize_int8", moe_ffn_quantize_int8(src.data_ptr(), rows, cols, q.data_ptr(), sc.data_ptr(), s))
        out[name + "_q"] = q
        out[name + "_scale"] = sc
    return out


def moe_ffn_quantize_mxfp4(w: int, rows: int, cols: int, codes: int, scales: int, stream: int) -> int:
    return lib().moe_ffn_quantize_mxfp4(_vp(w), int(rows), int(cols), _vp(codes), _vp(scales), _vp(stream))


def quantize_experts_mxfp4(w: dict) -> dict:
    """Adds the MXFP4 form of the experts (gate_up_f4/f4s, down_f4/f4s) to a dict of CUDA weight
    tensors, made on the device by moe_ffn_quantize_mxfp4."""
    import torch
    out = dict(w)
    s = torch.cuda.current_stream().cuda_stream
    for name, rows, cols in (("gate_up", N_EXPERTS * 2 * MOE_INTER, HIDDEN), ("down", N_EXPERTS * HIDDEN, MOE_INTER)):
        src = w[name]
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=src.device)
        sc = torch.empty((rows, cols // 32), dtype=torch.uint8, device=src.device)
        _check("moe_ffn_quantize_mxfp4",
               moe_ffn_quantize_mxfp4(src.data_ptr(), rows, cols, codes.data_ptr(), sc.data_ptr(), s))
        out[name + "_f4"] = codes
        out[name + "_f4s"] = sc
    return out


def moe_ffn_destroy(ctx: int) -> None:
    lib().moe_ffn_destroy(_vp(ctx))


def make_kv_config(q_heads: int, kv_heads: int, head_dim: int, page_size: int, n_pages: int, fmt: str,
                   max_tokens: int, max_seqs: int) -> moe_ffn_kv_config:
    return moe_ffn_kv_config(int(q_heads), int(kv_heads), int(head_dim), int(page_size), int(n_pages),
                             KV_FORMATS.get(fmt, -1), int(max_tokens), int(max_seqs))


def moe_ffn_kv_workspace_bytes(cfg: moe_ffn_kv_config) -> int:
    return lib().moe_ffn_kv_workspace_bytes(ctypes.byref(cfg))


def moe_ffn_kv_init(cfg: moe_ffn_kv_config, workspace: int, workspace_bytes: int, device: int) -> int:
    """Returns the handle (an int)."""
    h = _vp()
    _check("moe_ffn_kv_init", lib().moe_ffn_kv_init(ctypes.byref(h), ctypes.byref(cfg), _vp(workspace),
                                                     workspace_bytes, int(device)))
    return h.value


def moe_ffn_kv_write(kv: int, cache: moe_ffn_kv_cache, batch: moe_ffn_kv_batch, k: moe_ffn_kv_rows,
                     v: moe_ffn_kv_rows, stream: int) -> int:
    return lib().moe_ffn_kv_write(kv, cache, batch, k, v, stream)


def moe_ffn_kv_read(kv: int, cache: moe_ffn_kv_cache, batch: moe_ffn_kv_batch, k_out: int, v_out: int,
                    stream: int) -> int:
    return lib().moe_ffn_kv_read(kv, cache, batch, k_out, v_out, stream)


def moe_ffn_kv_attention(kv: int, cache: moe_ffn_kv_cache, batch: moe_ffn_kv_batch, q: moe_ffn_kv_rows, scale: float,
                         window: int, sinks: int, out: int, lse: int, stream: int) -> int:
    return lib().moe_ffn_kv_attention(kv, cache, batch, q, scale, window, sinks, out, lse, stream)


def moe_ffn_kv_device_status(kv: int, stream: int):
    w = ctypes.c_uint32(0)
    rc = lib().moe_ffn_kv_device_status(_vp(kv), _vp(stream), ctypes.byref(w))
    return rc, w.value


def moe_ffn_kv_destroy(kv: int) -> None:
    lib().moe_ffn_kv_destroy(_vp(kv))


def moe_ffn_kv_tree(kv: int, batch: moe_ffn_kv_batch, parents: int, masks: int, depth: int, stream: int) -> int:
    return lib().moe_ffn_kv_tree(kv, batch, parents, masks, depth, stream)


def moe_ffn_kv_tree_attention(kv: int, cache: moe_ffn_kv_cache, batch: moe_ffn_kv_batch, masks: int, q: moe_ffn_kv_rows,
                              scale: float, window: int, sinks: int, out: int, lse: int, stream: int) -> int:
    return lib().moe_ffn_kv_tree_attention(kv, cache, batch, masks, q, scale, window, sinks, out, lse, stream)


def moe_ffn_kv_keep(kv: int, caches, n_layers: int, batch: moe_ffn_kv_batch, nodes: int, nodes_stride: int,
                    nodes_cols: int, counts: int, new_len: int, stream: int) -> int:
    return lib().moe_ffn_kv_keep(kv, _by_ref(caches), n_layers, batch, nodes, nodes_stride, nodes_cols, counts, new_len, stream)


def moe_ffn_kv_reorder(kv: int, caches, n_layers: int, pages: int, pages_stride: int, pages_cols: int, lengths: int,
                       parents: int, users: int, beams: int, stream: int) -> int:
    return lib().moe_ffn_kv_reorder(kv, _by_ref(caches), n_layers, pages, pages_stride, pages_cols, lengths, parents, users, beams,
                                    stream)


def moe_ffn_block_norm(args: moe_ffn_norm, stream: int) -> int:
    return lib().moe_ffn_block_norm(_by_ref(args), stream)


def moe_ffn_rotary_table(freq, axis) -> list:
    """The pairs (turn, axis) of frequencies (radians per position) and axes."""
    n = len(freq)
    if len(axis) != n:
        raise ValueError("%d frequencies, %d axes" % (n, len(axis)))
    table = (moe_ffn_rotary_pair * max(n, 1))()
    _check("moe_ffn_rotary_table", lib().moe_ffn_rotary_table((ctypes.c_double * max(n, 1))(*freq),
                                                               (ctypes.c_int * max(n, 1))(*axis), n, table))
    return [(e.turn, e.axis) for e in table]


def moe_ffn_rotary_apply(args: moe_ffn_rotary, q: moe_ffn_kv_rows, k: moe_ffn_kv_rows, q_out: moe_ffn_kv_rows,
                         k_out: moe_ffn_kv_rows, stream: int) -> int:
    return lib().moe_ffn_rotary_apply(*(_by_ref(s) for s in (args, q, k, q_out, k_out)), stream)


def moe_ffn_beam_workspace_bytes(users: int, beams: int, vocab: int, count: int) -> int:
    return lib().moe_ffn_beam_workspace_bytes(int(users), int(beams), int(vocab), int(count))


def moe_ffn_beam_select(args: moe_ffn_beam, workspace: int, workspace_bytes: int, stream: int) -> int:
    return lib().moe_ffn_beam_select(_by_ref(args), workspace, workspace_bytes, stream)


# ------------------------------------------------------------------ torch convenience layer

def _field_specs():
    """Element type and element count of every weight field, as include/moe_ffn.h states them."""
    import torch
    H, E, K2, I, D = HIDDEN, N_EXPERTS, 2 * MOE_INTER, MOE_INTER, DENSE_INTER
    f32, bf16, i8, u8 = torch.float32, torch.bfloat16, torch.int8, torch.uint8
    spec = {"router_w": (f32, E * H), "router_norm_w": (f32, H), "per_expert_scale": (f32, E),
            "gate_up": (bf16, E * K2 * H), "down": (bf16, E * H * I), "dense_gate": (bf16, D * H),
            "dense_up": (bf16, D * H), "dense_down": (bf16, H * D),
            "gate_up_q": (i8, E * K2 * H), "gate_up_scale": (f32, E * K2), "down_q": (i8, E * H * I),
            "down_scale": (f32, E * H), "gate_up_f4": (u8, E * K2 * H // 2), "gate_up_f4s": (u8, E * K2 * H // 32),
            "down_f4": (u8, E * H * I // 2), "down_f4s": (u8, E * H * I // 32)}
    for name in ("pre_ff_ln", "pre_ff_ln_2", "post_ff_ln_1", "post_ff_ln_2", "post_ff_ln"):
        spec[name] = (f32, H)
    return spec


def _check_type_size(what, t, dtype, numel):
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.numel() != numel:
        raise ValueError("%s must hold %d elements, got %d" % (what, numel, t.numel()))


def _check_placement(what, t):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % what)


def weights_struct(w: dict) -> moe_ffn_weights:
    """A moe_ffn_weights whose fields point at the CUDA tensors of ``w`` (absent fields are NULL).

    Each present tensor must have the field's element type and element count (include/moe_ffn.h),
    so that the kernels never read past a tensor that is too small. Types and sizes of all fields
    are checked before any placement, so a wrong one is named first."""
    spec = _field_specs()
    present = [(f, w[f]) for f in WEIGHT_FIELDS + INT8_FIELDS + F4_FIELDS if w.get(f) is not None]
    for f, t in present:
        _check_type_size("weight " + f, t, *spec[f])
    s = moe_ffn_weights()
    for f, t in present:
        _check_placement("weight " + f, t)
        setattr(s, f, t.data_ptr())
    if "layer_scalar" not in w:
        raise ValueError("layer_scalar is required")
    s.layer_scalar = float(w["layer_scalar"])
    return s


def check_io(x, out=None) -> int:
    """Checks a forward's input (and output, if given): contiguous bf16 CUDA tensors of shape
    [T, 2816], the output the same shape as the input. Returns T."""
    import torch
    if x.dim() != 2 or x.shape[1] != HIDDEN:
        raise ValueError("x must have shape [T, %d], got %s" % (HIDDEN, tuple(x.shape)))
    T = x.shape[0]
    _check_type_size("x", x, torch.bfloat16, T * HIDDEN)
    if out is not None:
        if tuple(out.shape) != tuple(x.shape):
            raise ValueError("out must have the shape of x %s, got %s" % (tuple(x.shape), tuple(out.shape)))
        _check_type_size("out", out, torch.bfloat16, T * HIDDEN)
    _check_placement("x", x)
    if out is not None:
        _check_placement("out", out)
    return T


class MoeFFN:
    """One context with its workspace (a torch uint8 tensor on the device)."""

    def __init__(self, mode: int, max_tokens: int, device: int = 0, workspace=None):
        import torch
        self.cfg = make_config(mode, max_tokens)
        self.nbytes = moe_ffn_workspace_bytes(self.cfg)
        if self.nbytes == 0:
            raise ValueError("invalid configuration")
        self.device = int(device)
        if workspace is None:
            workspace = torch.empty(self.nbytes, dtype=torch.uint8, device="cuda:%d" % self.device)
        elif workspace.numel() < self.nbytes:
            raise ValueError("workspace too small")
        self.workspace = workspace
        self.ctx = moe_ffn_init(self.cfg, workspace.data_ptr(), workspace.numel(), self.device)

    def forward(self, x, weights, out=None, stream=None):
        import torch
        T = check_io(x, out)
        if out is None:
            out = torch.empty_like(x)
        ws = weights if isinstance(weights, moe_ffn_weights) else weights_struct(weights)
        s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
        _check("moe_ffn_forward", moe_ffn_forward(self.ctx, x.data_ptr(), T, ws, out.data_ptr(), s))
        return out

    def forward_shard(self, x, weights, expert_begin, expert_end, with_dense, stream=None):
        """One expert-parallel shard: (moe_partial, dense_out or None), fp32 [T, 2816] tensors."""
        import torch
        T = check_io(x)
        ws = weights if isinstance(weights, moe_ffn_weights) else weights_struct(weights)
        s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
        part = torch.empty((T, HIDDEN), dtype=torch.float32, device=x.device)
        dense = torch.empty((T, HIDDEN), dtype=torch.float32, device=x.device) if with_dense else None
        _check("moe_ffn_forward_shard",
               moe_ffn_forward_shard(self.ctx, x.data_ptr(), T, ws, expert_begin, expert_end, with_dense,
                                     part.data_ptr(), dense.data_ptr() if dense is not None else 0, s))
        return part, dense

    def finish_shards(self, x, weights, moe_sum, dense, out=None, stream=None):
        """The block's output from the summed shard partials (and the shared-MLP output)."""
        import torch
        T = check_io(x, out)
        for name, t in (("moe_sum", moe_sum), ("dense", dense)):
            if t is not None:
                _check_type_size(name, t, torch.float32, T * HIDDEN)
                _check_placement(name, t)
        if out is None:
            out = torch.empty_like(x)
        ws = weights if isinstance(weights, moe_ffn_weights) else weights_struct(weights)
        s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
        _check("moe_ffn_finish_shards",
               moe_ffn_finish_shards(self.ctx, x.data_ptr(), T, ws, moe_sum.data_ptr(),
                                     dense.data_ptr() if dense is not None else 0, out.data_ptr(), s))
        return out

    def views(self) -> moe_ffn_views:
        return moe_ffn_workspace_view(self.ctx)

    def status(self, stream=None):
        import torch
        s = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        return moe_ffn_device_status(self.ctx, s)

    def close(self):
        if self.ctx:
            moe_ffn_destroy(self.ctx)
            self.ctx = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _as_c_int(n: int) -> int:
    """The nearest window or number of sinks that a C int holds: no position lies further (ctypes would keep the
    lowest 32 bits), and a negative one is refused by the library."""
    return min(max(n, -1), 0x7fffffff)


class KVBatch:
    """The new tokens of a step, for PagedKV: device int32 tensors cu_q [n_seqs + 1] (first token row
    of each sequence), kv_len [n_seqs] (cached tokens, the new ones included) and pages [n_seqs, cols]
    (page ids; rows may be strided), and max_new, at least the largest number of new tokens of one
    sequence, by which the kernels are chosen: a loose one costs time. The tensors may be rewritten between calls (a captured graph reads them anew); their
    values are checked on the device."""

    def __init__(self, cu_q, kv_len, pages, max_new: int):
        import torch
        if kv_len.dim() != 1 or cu_q.dim() != 1 or pages.dim() != 2:
            raise ValueError("cu_q and kv_len must have one dimension and pages two")
        n = kv_len.shape[0]
        if cu_q.shape[0] != n + 1 or pages.shape[0] != n:
            raise ValueError("kv_len has %d sequences, cu_q %d and pages %d" % (n, cu_q.shape[0] - 1, pages.shape[0]))
        for name, t in (("cu_q", cu_q), ("kv_len", kv_len), ("pages", pages)):
            if t.dtype != torch.int32:
                raise ValueError("%s must be torch.int32, got %s" % (name, t.dtype))
        if max_new < 0:
            raise ValueError("max_new must not be negative")
        max_new = _as_c_int(max_new)
        for name, t in (("cu_q", cu_q), ("kv_len", kv_len)):
            _check_placement(name, t)
        cols = pages.shape[1]
        if not pages.is_cuda or (cols > 1 and pages.stride(1) != 1) or (n > 1 and pages.stride(0) < cols):
            raise ValueError("pages must be a CUDA tensor with contiguous rows")
        if kv_len.device != cu_q.device or pages.device != cu_q.device:
            raise ValueError("cu_q, kv_len and pages must be on one device")
        self.tensors = (cu_q, kv_len, pages)
        self.device = cu_q.device
        self.struct = moe_ffn_kv_batch(cu_q.data_ptr(), kv_len.data_ptr(), pages.data_ptr(),
                                       pages.stride(0) if n > 1 else cols, cols, n, 0, int(max_new))
        self._last = (-1, None)

    def of(self, n_tokens: int):
        """The C structure (by reference) for tensors of n_tokens token rows. One that was given out is not
        changed again: another thread's call may still be reading it."""
        last = self._last
        if last[0] != n_tokens:
            s = moe_ffn_kv_batch.from_buffer_copy(self.struct)
            s.n_tokens = n_tokens
            last = self._last = (n_tokens, ctypes.byref(s))
        return last[1]


class KVTree:
    """The trees of a batch as PagedKV.tree_attention reads them (PagedKV.tree makes it): masks, int32
    [tokens, 8], and depth, int32 [tokens], each node's number of ancestors: its position is the context's length
    plus that. Keep it as long as a graph that captured its attention."""

    def __init__(self, masks, depth, raw=None):
        self.masks, self.depth = masks, depth
        self._raw = raw  # the stream whose memory these are
        self.device = masks.device
        self.n_tokens = masks.shape[0]


class KVCache:
    """One layer's cache tensors, checked once (PagedKV.cache and PagedKV.new_cache make it). kind: the
    shape, type and device they were checked for; handles of another kind check them again and refuse."""

    def __init__(self, k, v, k_scale=None, v_scale=None, kind=None):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kind = kind
        self.struct = moe_ffn_kv_cache(*(t.data_ptr() if t is not None else None for t in (k, v, k_scale, v_scale)))
        self._ref = ctypes.byref(self.struct)
        self.packed = bytes(self.struct)


class PagedKV:
    """A paged key/value cache's shape, its handle and workspace; one serves all layers of that shape.

    fmt "bf16", or "e4m3" with an fp32 scale per token and head. Calls go to the current stream; a call
    on another stream than the last one's first waits for that one (not while a graph is captured:
    order the replays yourself, and keep the handle as long as the graph)."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_size: int, n_pages: int, fmt: str = "bf16",
                 max_tokens: int = 8192, max_seqs: int = 256, device: int = 0):
        import torch
        self.ctx = 0
        if fmt not in KV_FORMATS:
            raise ValueError("fmt must be one of %s, got %r" % (sorted(KV_FORMATS), fmt))
        self.cfg = make_kv_config(q_heads, kv_heads, head_dim, page_size, n_pages, fmt, max_tokens, max_seqs)
        self.nbytes = moe_ffn_kv_workspace_bytes(self.cfg)
        if self.nbytes == 0:
            raise ValueError("invalid configuration")
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        self.shape = (int(n_pages), self.kv_heads, int(page_size), self.head_dim)
        self.fmt = fmt
        self.dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
        self.default_scale = self.head_dim ** -0.5
        self.device = torch.device("cuda", int(device))
        self._kind = (self.shape, self.dtype, self.device)
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=self.device)
        self.ctx = moe_ffn_kv_init(self.cfg, self.workspace.data_ptr(), self.nbytes, int(device))
        self._handle = _vp(self.ctx)
        self._last = self._last_raw = None

    def new_cache(self) -> KVCache:
        """A zeroed cache of one layer."""
        import torch
        k, v = (torch.zeros(self.shape, dtype=self.dtype, device=self.device) for _ in range(2))
        if self.fmt == "bf16":
            return KVCache(k, v, kind=self._kind)
        return KVCache(k, v, *(torch.zeros(self.shape[:3], device=self.device) for _ in range(2)), kind=self._kind)

    def cache(self, k, v, k_scale=None, v_scale=None) -> KVCache:
        """A cache over existing tensors, checked against this shape."""
        import torch
        wanted = [("k", k, self.dtype, self.shape), ("v", v, self.dtype, self.shape)]
        if self.fmt == "e4m3":
            wanted += [(n, t, torch.float32, self.shape[:3]) for n, t in (("k_scale", k_scale), ("v_scale", v_scale))]
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        for name, t, dtype, shape in wanted:
            if t is None:
                raise ValueError("%s is required" % name)
            if t.dtype != dtype or tuple(t.shape) != shape:
                raise ValueError("%s must be %s of shape %s, got %s of shape %s" % (name, dtype, shape, t.dtype,
                                                                                    tuple(t.shape)))
        for name, t, _, _ in wanted:
            _check_placement(name, t)
            if t.device != self.device:
                raise ValueError("%s must be on %s" % (name, self.device))
        return KVCache(k, v, k_scale, v_scale, self._kind)

    def _rows(self, what, t, heads):
        import torch
        if t.dtype != torch.bfloat16:
            raise ValueError("%s must be torch.bfloat16, got %s" % (what, t.dtype))
        shape = t.shape
        if len(shape) != 3 or shape[1] != heads or shape[2] != self.head_dim:
            raise ValueError("%s must have shape [tokens, %d, %d], got %s" % (what, heads, self.head_dim, tuple(shape)))
        if t.device != self.device:
            raise ValueError("%s must be on %s" % (what, self.device))
        ts, hs, es = t.stride()
        # A dimension of one element has no stride that matters.
        if shape[0] <= 1:
            ts = 0
        if heads == 1:
            hs = 0
        if es != 1 or ts % 8 or hs % 8:
            raise ValueError("%s must have a contiguous last dimension and strides that are multiples of 8" % what)
        return moe_ffn_kv_rows(t.data_ptr(), ts, hs)

    def _begin(self, cache, batch):
        """The cache's structure and the stream of a call, ordered after the handle's last one."""
        if not isinstance(cache, KVCache):
            cache = self.cache(**cache)
        elif cache.kind != self._kind:
            cache = self.cache(cache.k, cache.v, cache.k_scale, cache.v_scale)
        return cache._ref, self._stream(batch)

    def _stream(self, batch=None):
        import torch
        if batch is not None and batch.device != self.device:
            raise ValueError("the batch must be on %s" % self.device)
        raw = torch._C._cuda_getCurrentRawStream(self.device.index)
        if raw != self._last_raw and not torch.cuda.is_current_stream_capturing():
            stream = torch.cuda.current_stream(self.device)
            if self._last is not None:
                stream.wait_stream(self._last)
            self.workspace.record_stream(stream)  # dropped early, it stays until the stream is done with it
            self._last, self._last_raw = stream, raw
        return raw

    def write(self, cache, batch: KVBatch, k, v) -> None:
        """Writes the new tokens' keys and values, bf16 [tokens, kv_heads, head_dim] each, into `cache`
        (a KVCache, or a dict of its tensors)."""
        kr, vr = self._rows("k", k, self.kv_heads), self._rows("v", v, self.kv_heads)
        if k.shape[0] != v.shape[0]:
            raise ValueError("k has %d tokens, v %d" % (k.shape[0], v.shape[0]))
        c, s = self._begin(cache, batch)
        _check("moe_ffn_kv_write", moe_ffn_kv_write(self._handle, c, batch.of(k.shape[0]), kr, vr, s))

    def read(self, cache, batch: KVBatch, n_tokens=None):
        """The batch's tokens read back: (k, v), bf16 [tokens, kv_heads, head_dim]. n_tokens: the token
        rows of the batch, cu_q's last value (which is read from the device if it is not given)."""
        import torch
        if n_tokens is None:
            n_tokens = int(batch.tensors[0][-1])
        k, v = (torch.empty((n_tokens, self.kv_heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
                for _ in range(2))
        c, s = self._begin(cache, batch)
        _check("moe_ffn_kv_read",
               moe_ffn_kv_read(self._handle, c, batch.of(n_tokens), k.data_ptr(), v.data_ptr(), s))
        return k, v

    def attention(self, cache, batch: KVBatch, q, window: int = 0, sinks: int = 0, scale=None, out=None):
        """Attention of the new tokens' queries, bf16 [tokens, q_heads, head_dim], over the cache, causal,
        with an optional sliding window and first positions that stay visible: (out, lse), bf16 like q
        (contiguous) and fp32 [tokens, q_heads]. scale: head_dim ** -0.5 if not given."""
        return self._attend(cache, batch, None, q, window, sinks, scale, out)

    def _attend(self, cache, batch, tree, q, window, sinks, scale, out):
        import torch
        qr = self._rows("q", q, self.q_heads)
        T = q.shape[0]
        if out is None:
            out = torch.empty((T, self.q_heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
        else:
            if tuple(out.shape) != tuple(q.shape):
                raise ValueError("out must have the shape of q %s, got %s" % (tuple(q.shape), tuple(out.shape)))
            _check_type_size("out", out, torch.bfloat16, q.numel())
            _check_placement("out", out)
        lse = torch.empty((T, self.q_heads), dtype=torch.float32, device=self.device)
        c, s = self._begin(cache, batch)
        scale = self.default_scale if scale is None else scale
        window, sinks = _as_c_int(window), _as_c_int(sinks)
        if tree is None:
            _check("moe_ffn_kv_attention", moe_ffn_kv_attention(self._handle, c, batch.of(T), qr, scale, window, sinks,
                                                                out.data_ptr(), lse.data_ptr(), s))
        else:
            if s != tree._raw and tree._raw is not None and not torch.cuda.is_current_stream_capturing():
                tree.masks.record_stream(torch.cuda.current_stream(self.device))  # dropped early, they stay until it is done
            _check("moe_ffn_kv_tree_attention",
                   moe_ffn_kv_tree_attention(self._handle, c, batch.of(T), tree.masks.data_ptr(), qr, scale, window, sinks,
                                             out.data_ptr(), lse.data_ptr(), s))
        return out, lse

    def _ids(self, what, t, *shape):
        import torch
        if t.dtype != torch.int32 or t.shape != shape:
            raise ValueError("%s must be torch.int32 of shape %s, got %s of shape %s" % (what, list(shape), t.dtype,
                                                                                         list(t.shape)))
        if t.device != self.device or not t.is_contiguous():
            raise ValueError("%s must be a contiguous tensor on %s" % (what, self.device))

    def _layers(self, caches):
        """Several layers' caches as an array of structures, packed."""
        if isinstance(caches, (KVCache, dict)):
            caches = [caches]
        packed = []
        for c in caches:
            if not isinstance(c, KVCache):
                c = self.cache(**c)
            elif c.kind != self._kind:
                c = self.cache(c.k, c.v, c.k_scale, c.v_scale)
            packed.append(c.packed)
        return b"".join(packed), len(packed)

    def tree(self, batch: KVBatch, parents) -> KVTree:
        """The trees of a batch whose new tokens are drafted ones: parents, int32 [tokens], gives each node's parent
        among its sequence's nodes (an earlier one), or -1 where it follows the context. At most 256 nodes to a
        sequence. One serves all layers."""
        import torch
        if parents.dim() != 1:
            raise ValueError("parents must have one dimension, got shape %s" % (list(parents.shape),))
        T = parents.shape[0]
        self._ids("parents", parents, T)
        masks = torch.empty((T, 8), dtype=torch.int32, device=self.device)
        depth = torch.empty((T,), dtype=torch.int32, device=self.device)
        s = self._stream(batch)
        _check("moe_ffn_kv_tree", moe_ffn_kv_tree(self._handle, batch.of(T), parents.data_ptr(), masks.data_ptr(),
                                                  depth.data_ptr(), s))
        return KVTree(masks, depth, s)

    def tree_attention(self, cache, batch: KVBatch, tree: KVTree, q, window: int = 0, sinks: int = 0, scale=None, out=None):
        """Attention of drafted tokens' queries, bf16 [tokens, q_heads, head_dim], over the cache, which holds their
        keys and values: a node sees the context, its ancestors and itself (window and sinks by positions).
        Returns (out, lse) as attention does."""
        if tree.device != self.device or tree.n_tokens != q.shape[0]:
            raise ValueError("the tree has %d tokens on %s, q %d on %s" % (tree.n_tokens, tree.device, q.shape[0], self.device))
        return self._attend(cache, batch, tree, q, window, sinks, scale, out)

    def keep(self, caches, batch: KVBatch, nodes, counts):
        """Keeps one path of each tree of `batch` in all layers' `caches` (a list, or one): the nodes
        nodes[b, i], i < counts[b], ascending, move to the slots after the context. nodes: int32
        [sequences, any], counts: int32 [sequences]. Returns the cached tokens that remain, int32 [sequences]."""
        import torch
        n = batch.tensors[1].shape[0]
        if nodes.dim() != 2:
            raise ValueError("nodes must have two dimensions, got shape %s" % (list(nodes.shape),))
        self._ids("nodes", nodes, n, nodes.shape[1])
        self._ids("counts", counts, n)
        layers, n_layers = self._layers(caches)
        new_len = torch.empty((n,), dtype=torch.int32, device=self.device)
        s = self._stream(batch)
        _check("moe_ffn_kv_keep",
               moe_ffn_kv_keep(self._handle, layers, n_layers, batch.of(self.cfg.max_tokens), nodes.data_ptr(), nodes.shape[1],
                               nodes.shape[1], counts.data_ptr(), new_len.data_ptr(), s))
        return new_len

    def reorder(self, caches, pages, lengths, parents) -> None:
        """The states of beams follow their parents, int32 [users, beams], in all layers' `caches` (a list, or one).
        pages: the page table, int32 [users * beams, cols] with contiguous rows, changed in place; lengths: int32
        [users], the cached tokens of each of a user's beams. Full pages are shared through the table; of
        the page under way, which with those after it is each beam's own, the tokens so far are copied."""
        import torch
        if parents.dim() != 2:
            raise ValueError("parents must have two dimensions, got shape %s" % (list(parents.shape),))
        users, beams = parents.shape
        self._ids("parents", parents, users, beams)
        self._ids("lengths", lengths, users)
        if pages.dtype != torch.int32 or pages.dim() != 2 or pages.shape[0] != users * beams:
            raise ValueError("pages must be torch.int32 of shape [%d, columns], got %s of shape %s" % (
                users * beams, pages.dtype, list(pages.shape)))
        cols = pages.shape[1]
        stride = pages.stride(0) if pages.shape[0] > 1 else cols
        if pages.device != self.device or (cols > 1 and pages.stride(1) != 1) or stride < cols:
            raise ValueError("pages must be a tensor with contiguous rows on %s" % self.device)
        layers, n_layers = self._layers(caches)
        s = self._stream()
        _check("moe_ffn_kv_reorder",
               moe_ffn_kv_reorder(self._handle, layers, n_layers, pages.data_ptr(), stride, cols, lengths.data_ptr(),
                                  parents.data_ptr(), users, beams, s))

    def status(self, stream=None):
        import torch
        s = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        return moe_ffn_kv_device_status(self.ctx, s)

    def close(self):
        if self.ctx:
            moe_ffn_kv_destroy(self.ctx)
            self.ctx = 0
            self._handle = None  # calls are refused from here on

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _launch(call, device, *args):
    """A call without a handle, on the current stream of its tensors' device."""
    import torch
    raw = torch._C._cuda_getCurrentRawStream(device.index)
    if torch._C._cuda_getDevice() == device.index:
        return call(*args, raw)
    with torch.cuda.device(device):
        return call(*args, raw)


def _norm_rows(what, t, shape, device, bf16):
    """Address and row stride of bf16 rows."""
    if t.dtype != bf16 or t.shape != shape:
        raise ValueError("%s must be torch.bfloat16 of shape %s, got %s of shape %s" % (what, list(shape), t.dtype,
                                                                                        list(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s" % (what, device))
    step, one = t.stride()
    if shape[0] <= 1:
        step = shape[1]
    if one != 1 or step % 8:
        raise ValueError("%s must have contiguous rows, a multiple of 8 elements apart" % what)
    return t.data_ptr(), step


def _norm_weight(what, w, H, device, f32):
    if w.dtype != f32 or w.numel() != H:
        _check_type_size(what, w, f32, H)
    if w.device != device or not w.is_contiguous():
        raise ValueError("%s must be a contiguous tensor on %s" % (what, device))
    return w.data_ptr()


def block_norm(x, block=None, post=None, gate=None, scale: float = 1.0, pre=None, eps: float = 1e-6, out=None, normed=None):
    """The norm after one block and the one before the next, with the gated residual between them:

        y = scale * (x + gate * N(block; post)),  n = N(y; pre),  N(v; w) = v / rms(v) * (1 + w)

    x, block and gate: bf16 [tokens, hidden] (rows may be strided, a gate for all rows expanded); post and pre: fp32
    [hidden]. Without a block y is scale * x; without post the block is added without a norm. Returns (y, n), bf16; n
    is None without pre, and y is None where it would be x itself (no block, scale 1, no out). out and normed: where y
    and n go, x or block themselves if wished."""
    import torch
    bf16, f32, shape = torch.bfloat16, torch.float32, x.shape
    if len(shape) != 2:
        raise ValueError("x must have two dimensions, got shape %s" % (list(shape),))
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    T, H = shape
    device = x.device
    if block is None and (post is not None or gate is not None):
        raise ValueError("post and gate need a block")
    if pre is None and normed is not None:
        raise ValueError("normed needs pre")
    xp, xs = _norm_rows("x", x, shape, device, bf16)
    bp, bs = (0, 0) if block is None else _norm_rows("block", block, shape, device, bf16)
    gp, gs = (0, 0) if gate is None else _norm_rows("gate", gate, shape, device, bf16)
    post_p = 0 if post is None else _norm_weight("post", post, H, device, f32)
    pre_p = 0 if pre is None else _norm_weight("pre", pre, H, device, f32)
    yp, ys = 0, 0
    if out is not None:
        yp, ys = _norm_rows("out", out, shape, device, bf16)
    elif block is not None or scale != 1.0 or pre is None:
        out = torch.empty(shape, dtype=bf16, device=device)
        yp, ys = out.data_ptr(), H
    np_, ns = 0, 0
    if normed is not None:
        np_, ns = _norm_rows("normed", normed, shape, device, bf16)
    elif pre is not None:
        normed = torch.empty(shape, dtype=bf16, device=device)
        np_, ns = normed.data_ptr(), H
    _check("moe_ffn_block_norm",
           _launch(lib().moe_ffn_block_norm, device,
                   _PACK_NORM(xp, bp, gp, post_p, pre_p, yp, np_, xs, bs, gs, ys, ns, scale, eps, T, H)))
    return out, normed


class Rotary:
    """Rotary positions with one or several axes. freqs: each pair's radians per position; axes: the axis whose
    position turns it (all 0 if not given). Pair i of a head is (i, pairs + i), or (2i, 2i + 1) where interleaved;
    elements after the pairs stay as they are. scale multiplies the turned elements. Keep the object as long as a graph
    that captured it."""

    def __init__(self, freqs, axes=None, interleaved: bool = False, scale: float = 1.0, device: int = 0):
        import torch
        freqs = [float(f) for f in freqs]
        axes = [0] * len(freqs) if axes is None else [int(i) for i in axes]
        if not freqs or len(freqs) % 4 or len(freqs) > ROTARY_MAX_PAIRS:
            raise ValueError("the number of pairs must be a multiple of 4 up to %d, got %d" % (ROTARY_MAX_PAIRS, len(freqs)))
        rows = moe_ffn_rotary_table(freqs, axes)
        signed = [[v - (1 << 64) if v >= 1 << 63 else v for v in row] for row in rows]
        self.device = torch.device("cuda", int(device))
        self.pairs, self.axes = len(freqs), max(axes) + 1
        self.interleaved, self.scale = bool(interleaved), float(scale)
        self.table = torch.tensor(signed, dtype=torch.int64).to(self.device)
        self._table = self.table.data_ptr()
        self._last_raw = None

    def _rows(self, what, t, T, D, bf16):
        """A tensor's address and strides, packed, and its heads."""
        shape = t.shape
        if t.dtype != bf16 or len(shape) != 3 or shape[0] != T or shape[2] != D:
            raise ValueError("%s must be torch.bfloat16 of shape [%d, heads, %d], got %s of shape %s" % (what, T, D, t.dtype,
                                                                                                         list(shape)))
        if t.device != self.device:
            raise ValueError("%s must be on %s" % (what, self.device))
        heads = shape[1]
        ts, hs, es = t.stride()
        # A dimension of one element has no stride that matters.
        if T <= 1:
            ts = 0
        if heads <= 1:
            hs = 0
        if es != 1 or ts % 8 or hs % 8:
            raise ValueError("%s must have a contiguous last dimension and strides that are multiples of 8" % what)
        return _PACK_ROWS(t.data_ptr(), ts, hs), heads

    def apply(self, q, k, positions, inverse: bool = False, inplace: bool = False):
        """Turns q and k, bf16 [tokens, heads, width] each (any strides of 8 elements; k may be None), by positions, int32
        [axes, tokens] (or [tokens] for one axis). Returns (q, k), new tensors or, inplace, the given ones. inverse turns
        back, which is also the gradient's way."""
        import torch
        bf16, device = torch.bfloat16, self.device
        if q.dim() != 3:
            raise ValueError("q must have three dimensions, got shape %s" % (list(q.shape),))
        T, _, D = q.shape
        at = positions.shape
        axes, n = at if len(at) == 2 else (1, at[0]) if len(at) == 1 else (0, 0)
        if positions.dtype != torch.int32 or axes < self.axes or n != T:
            raise ValueError("positions must be torch.int32 of shape [%d, %d], got %s of shape %s" % (
                self.axes, T, positions.dtype, list(at)))
        steps = positions.stride()
        if positions.device != device or (T > 1 and steps[-1] != 1):
            raise ValueError("positions must have contiguous rows on %s" % device)
        q_rows, q_heads = self._rows("q", q, T, D, bf16)
        k_rows, k_heads = (None, 0) if k is None else self._rows("k", k, T, D, bf16)
        q_to, k_to = q_rows, k_rows
        if not inplace:
            q = torch.empty((T, q_heads, D), dtype=bf16, device=device)
            q_to = _PACK_ROWS(q.data_ptr(), q_heads * D if T > 1 else 0, D if q_heads > 1 else 0)
            if k is not None:
                k = torch.empty((T, k_heads, D), dtype=bf16, device=device)
                k_to = _PACK_ROWS(k.data_ptr(), k_heads * D if T > 1 else 0, D if k_heads > 1 else 0)
        raw = torch._C._cuda_getCurrentRawStream(device.index)
        if raw != self._last_raw and not torch.cuda.is_current_stream_capturing():
            self.table.record_stream(torch.cuda.current_stream(device))  # dropped early, it stays until the stream is done with it
            self._last_raw = raw
        a = _PACK_ROTARY(self._table, positions.data_ptr(), steps[0] if self.axes > 1 else 0, self.scale, self.pairs, self.axes,
                         self.interleaved, inverse, T, D, q_heads, k_heads)
        _check("moe_ffn_rotary_apply", _launch(lib().moe_ffn_rotary_apply, device, a, q_rows, k_rows, q_to, k_to))
        return q, k


class BeamSearch:
    """The selection of a beam search, with its workspace: of each user's beams * vocab continuations the `count` best.
    Calls share the workspace: on another stream than the last one's, a call first waits for that one (not while
    a graph is captured: order the replays yourself, and keep the object as long as the graph)."""

    def __init__(self, users: int, beams: int, vocab: int, count: int, device: int = 0):
        import torch
        self.users, self.beams, self.vocab, self.count = int(users), int(beams), int(vocab), int(count)
        self.nbytes = moe_ffn_beam_workspace_bytes(self.users, self.beams, self.vocab, self.count)
        if self.nbytes == 0:
            raise ValueError("invalid configuration")
        self.device = torch.device("cuda", int(device))
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=self.device)
        # It may be memory that work still queued on this stream writes; the first call may come on another one, or be
        # captured, and then waits for nothing. (Allocated within a capture it is the graph's own.)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.device).synchronize()
        self._workspace = self.workspace.data_ptr()
        self._shapes = tuple(torch.Size(t) for t in ((self.users * self.beams, self.vocab), (self.users, self.beams, self.vocab),
                                                     (self.users, self.beams)))
        self._last = self._last_raw = None

    def select(self, logits, scores, finished=None, end_token: int = 0):
        """logits: bf16 or fp32 [users * beams, vocab] (or [users, beams, vocab]), rows may be strided; scores: fp32
        [users, beams], the beams' sums so far (-infinity: no such beam); finished: bool [users, beams], whose only
        continuation is end_token with the same score. Returns (scores, beams, tokens), each [users, count], best first;
        beam and token are -1 where there is no further continuation."""
        import torch
        U, K, V, C = self.users, self.beams, self.vocab, self.count
        device, shape, steps = self.device, logits.shape, logits.stride()
        wide = logits.dtype == torch.float32
        if not wide and logits.dtype != torch.bfloat16:
            raise ValueError("logits must be torch.bfloat16 or torch.float32, got %s" % logits.dtype)
        if shape == self._shapes[0]:
            stride = steps[0]
        elif shape == self._shapes[1]:
            if U > 1 and K > 1 and steps[0] != K * steps[1]:
                raise ValueError("logits' rows must lie at one stride")
            stride = steps[1] if K > 1 else steps[0]
        else:
            raise ValueError("logits must have shape [%d, %d], got %s" % (U * K, V, list(shape)))
        if V > 1 and steps[-1] != 1:
            raise ValueError("logits must have contiguous rows")
        for name, t, dtype in (("scores", scores, torch.float32), ("finished", finished, torch.bool)):
            if t is None and name == "finished":
                continue
            if t.dtype != dtype or t.shape != self._shapes[2] or not t.is_contiguous():
                raise ValueError("%s must be contiguous, %s of shape [%d, %d], got %s of shape %s" % (name, dtype, U, K, t.dtype,
                                                                                                      list(t.shape)))
            if t.device != device:
                raise ValueError("%s must be on %s" % (name, device))
        if logits.device != device:
            raise ValueError("logits must be on %s" % device)
        out = torch.empty((U, C), dtype=torch.float32, device=device)
        beams = torch.empty((U, C), dtype=torch.int32, device=device)
        tokens = torch.empty((U, C), dtype=torch.int32, device=device)
        a = _PACK_BEAM(logits.data_ptr(), stride if U * K > 1 else V, scores.data_ptr(),
                       0 if finished is None else finished.data_ptr(), out.data_ptr(), beams.data_ptr(), tokens.data_ptr(), wide,
                       end_token, U, K, V, C)
        raw = torch._C._cuda_getCurrentRawStream(device.index)
        if raw != self._last_raw and not torch.cuda.is_current_stream_capturing():
            stream = torch.cuda.current_stream(device)
            if self._last is not None:
                stream.wait_stream(self._last)
            self.workspace.record_stream(stream)  # dropped early, it stays until the stream is done with it
            self._last, self._last_raw = stream, raw
        _check("moe_ffn_beam_select", _launch(lib().moe_ffn_beam_select, device, a, self._workspace, self.nbytes))
        return out, beams, tokens


def view_tensor(ptr: int, shape, dtype, device: int = 0):
    """A torch tensor aliasing device memory at ``ptr`` (for reading the workspace views)."""
    import torch
    n = 1
    for s in shape:
        n *= s
    if n == 0:
        return torch.empty(shape, dtype=dtype, device="cuda:%d" % device)
    nbytes = n * torch.empty((), dtype=dtype).element_size()

    class _Holder:
        __cuda_array_interface__ = {
            "shape": (nbytes,), "typestr": "|u1", "data": (ptr, False), "version": 3, "strides": None,
        }

    raw = torch.as_tensor(_Holder(), device="cuda:%d" % device)
    return raw.view(dtype).view(*shape)
