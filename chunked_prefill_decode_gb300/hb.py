"""ctypes binding of libhb.so (the C ABI declared in include/hb.h).

Argument marshalling only: every function here turns torch tensors / numpy
arrays into the pointers and sizes the C calls take, calls them, and raises
HbError on a non-zero status.  All computation runs in the library's CUDA
kernels; there is no fallback, and loading fails loudly when the library is
missing.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhb.so")
_lib = None

HB_OK = 0
HB_NUM_KERNEL_IDS = 3
KERNEL_NAMES = ("kv_append", "attention", "linear")

STATUS_NAMES = {
    0: "HB_OK", 1: "HB_ERR_INVALID_ARG", 2: "HB_ERR_SHAPE", 3: "HB_ERR_UNSUPPORTED",
    4: "HB_ERR_WORKSPACE", 5: "HB_ERR_CUDA", 6: "HB_ERR_DEVICE_INDEX",
    7: "HB_ERR_TIMEOUT", 8: "HB_ERR_OUT_OF_PAGES",
}


class HbError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class HbBatch(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("total_q", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("sliding_window", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("cu_q_len", ctypes.c_void_p),
        ("context_len", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
    ]


EXPORTED = (
    "hb_last_error", "hb_status_string", "hb_kv_append", "hb_plan", "hb_attention",
    "hb_attention_new_kv",
    "hb_check", "hb_timing_enable", "hb_timing_read", "hb_launch_count",
    "hb_builder_create", "hb_builder_destroy", "hb_builder_add_request",
    "hb_builder_step", "hb_builder_complete", "hb_builder_counts",
    "hb_builder_free_list", "hb_builder_last_error", "hb_decode_attention_noalloc",
    "hb_selftest_wait_timeout", "hb_selftest_flag_timeout", "hb_linear", "hb_linear_workspace_size",
    "hb_timing_durations", "hb_step_layout", "hb_step_slot_create", "hb_step_slot_destroy",
    "hb_step_slot_sync", "hb_step", "hb_kv8_append", "hb_kv8_plan", "hb_kv8_attention",
    "hb_pages_assign", "hb_pages_release", "hb_norm", "hb_rope_phases", "hb_rope",
    "hb_adapters_plan", "hb_adapters",
)

LINEAR_STORE, LINEAR_GATED, LINEAR_RESIDUAL = 0, 1, 2


class HbStepBuffers(ctypes.Structure):
    _fields_ = [("h_in", ctypes.c_void_p), ("d_in", ctypes.c_void_p),
                ("h_out", ctypes.c_void_p), ("d_out", ctypes.c_void_p),
                ("h_plan", ctypes.c_void_p), ("plan_bytes", ctypes.c_size_t),
                ("d_workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


HB_STEP_SECTIONS = 6


class HbLinearOut(ctypes.Structure):
    _fields_ = [("y", ctypes.c_void_p * 3), ("cols", ctypes.c_int32 * 3)]


class HbNormArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("rows", "width", "stream_type", "reserved")]
                + [(n, ctypes.c_void_p) for n in ("x", "y", "gate", "w_post", "w_pre", "x_out", "z")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "y_stride", "gate_stride", "x_out_stride", "z_stride")]
                + [(n, ctypes.c_float) for n in ("eps", "residual_scale", "branch_scale", "weight_offset")])


class HbRopeParams(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float),
                ("eps", ctypes.c_float), ("phases", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p)]


ROPE_SCALINGS = ("none", "linear", "base", "parts")


class HbAdapterPool(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_adapters", "max_rank", "K", "N", "slices")]
                + [(n, ctypes.c_void_p) for n in ("a", "b", "rank", "scale")])


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libhb.so (raising if it has not been built) and declare its calls."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    P = ctypes.POINTER
    L.hb_last_error.restype = ctypes.c_char_p
    L.hb_last_error.argtypes = []
    L.hb_builder_last_error.restype = ctypes.c_char_p
    L.hb_builder_last_error.argtypes = []
    L.hb_status_string.restype = ctypes.c_char_p
    L.hb_status_string.argtypes = [ctypes.c_int]
    L.hb_kv_append.restype = ctypes.c_int
    L.hb_kv_append.argtypes = [P(HbBatch), vp, vp, vp, vp, vp]
    L.hb_plan.restype = ctypes.c_int
    L.hb_plan.argtypes = [P(HbBatch), vp, vp, i32, vp, P(sz), vp, P(sz), vp]
    L.hb_attention.restype = ctypes.c_int
    L.hb_attention.argtypes = [P(HbBatch), vp, vp, vp, vp, ctypes.c_float, vp, vp, vp]
    L.hb_attention_new_kv.restype = ctypes.c_int
    L.hb_attention_new_kv.argtypes = [P(HbBatch), vp, vp, vp, vp, vp, vp, ctypes.c_float, vp,
                                      vp, vp]
    L.hb_decode_attention_noalloc.restype = ctypes.c_int
    L.hb_decode_attention_noalloc.argtypes = [P(HbBatch), vp, vp, vp, vp, vp, ctypes.c_float,
                                              vp, vp]
    L.hb_linear.restype = ctypes.c_int
    L.hb_linear.argtypes = [vp, vp, i32, i32, i32, i32, P(HbLinearOut), vp, sz, vp]
    L.hb_linear_workspace_size.restype = sz
    L.hb_linear_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.hb_selftest_wait_timeout.restype = ctypes.c_int
    L.hb_selftest_wait_timeout.argtypes = [vp]
    L.hb_selftest_flag_timeout.restype = ctypes.c_int
    L.hb_selftest_flag_timeout.argtypes = [vp]
    L.hb_check.restype = ctypes.c_int
    L.hb_check.argtypes = [vp]
    L.hb_timing_enable.restype = ctypes.c_int
    L.hb_timing_enable.argtypes = [i32]
    L.hb_timing_read.restype = ctypes.c_int
    L.hb_timing_read.argtypes = [P(ctypes.c_double), P(i32)]
    L.hb_timing_durations.restype = ctypes.c_int
    L.hb_timing_durations.argtypes = [i32, P(ctypes.c_float), i32, P(i32)]
    L.hb_step_layout.restype = ctypes.c_int
    L.hb_step_layout.argtypes = [P(HbBatch), P(sz), P(sz)]
    L.hb_step_slot_create.restype = ctypes.c_int
    L.hb_step_slot_create.argtypes = [P(vp)]
    L.hb_step_slot_destroy.restype = None
    L.hb_step_slot_destroy.argtypes = [vp]
    L.hb_step_slot_sync.restype = ctypes.c_int
    L.hb_step_slot_sync.argtypes = [vp]
    L.hb_step.restype = ctypes.c_int
    L.hb_step.argtypes = [P(HbBatch), vp, vp, i32, vp, P(HbStepBuffers), vp, vp,
                          ctypes.c_float, vp, vp, vp]
    L.hb_kv8_append.restype = ctypes.c_int
    L.hb_kv8_append.argtypes = [P(HbBatch), vp, vp, vp, vp, vp, vp, vp]
    L.hb_kv8_plan.restype = ctypes.c_int
    L.hb_kv8_plan.argtypes = [P(HbBatch), vp, vp, i32, vp, P(sz), vp, P(sz), vp]
    L.hb_kv8_attention.restype = ctypes.c_int
    L.hb_kv8_attention.argtypes = [P(HbBatch), vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp]
    L.hb_pages_assign.restype = ctypes.c_int
    L.hb_pages_assign.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.hb_pages_release.restype = ctypes.c_int
    L.hb_pages_release.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.hb_norm.restype = ctypes.c_int
    L.hb_norm.argtypes = [vp, vp]
    L.hb_rope_phases.restype = ctypes.c_int
    L.hb_rope_phases.argtypes = [i32, ctypes.c_double, i32] + [ctypes.c_double] * 4 + [vp]
    L.hb_rope.restype = ctypes.c_int
    L.hb_rope.argtypes = [P(HbBatch), P(HbRopeParams), vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp]
    L.hb_adapters_plan.restype = ctypes.c_int
    L.hb_adapters_plan.argtypes = [i32, i32, vp, vp, i32, i32, i32, vp, P(sz), vp, P(sz), vp]
    L.hb_adapters.restype = ctypes.c_int
    L.hb_adapters.argtypes = [P(HbAdapterPool), vp, vp, vp, vp, vp, vp]
    L.hb_launch_count.restype = i64
    L.hb_launch_count.argtypes = []
    L.hb_builder_create.restype = ctypes.c_int
    L.hb_builder_create.argtypes = [i32, i32, i32, i32, vp, P(vp)]
    L.hb_builder_destroy.restype = None
    L.hb_builder_destroy.argtypes = [vp]
    L.hb_builder_add_request.restype = ctypes.c_int
    L.hb_builder_add_request.argtypes = [vp, i64, i32, i32]
    L.hb_builder_step.restype = ctypes.c_int
    L.hb_builder_step.argtypes = [vp, i32, P(i32), vp, vp, vp, vp, vp, P(i32)]
    L.hb_builder_complete.restype = ctypes.c_int
    L.hb_builder_complete.argtypes = [vp, i32, P(i32), vp]
    L.hb_builder_counts.restype = ctypes.c_int
    L.hb_builder_counts.argtypes = [vp, P(i32), P(i32), P(i32)]
    L.hb_builder_free_list.restype = ctypes.c_int
    L.hb_builder_free_list.argtypes = [vp, i32, P(i32), vp]
    _lib = L
    return L


def _check(status, builder=False):
    if status != HB_OK:
        L = load()
        msg = (L.hb_builder_last_error() if builder else L.hb_last_error()) or b""
        raise HbError(status, msg.decode(errors="replace"))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return ctypes.c_void_p(t.data_ptr()) if t.numel() else None
    if isinstance(t, np.ndarray):
        return t.ctypes.data_as(ctypes.c_void_p)
    return t


def _stream(stream):
    if stream is None:
        if torch.cuda.is_available():
            return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        return None
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def make_batch(num_seqs, total_q, max_pages_per_seq, num_pages, num_q_heads,
               num_kv_heads, head_dim, cu_q_len, context_len, block_table,
               page_size=16, sliding_window=0) -> HbBatch:
    """hb_batch over device int32 tensors (kept alive by the caller)."""
    for name, t in (("cu_q_len", cu_q_len), ("context_len", context_len),
                    ("block_table", block_table)):
        if t is not None and isinstance(t, torch.Tensor):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor")
    b = HbBatch()
    b.num_seqs, b.total_q = int(num_seqs), int(total_q)
    b.max_pages_per_seq, b.num_pages = int(max_pages_per_seq), int(num_pages)
    b.num_q_heads, b.num_kv_heads = int(num_q_heads), int(num_kv_heads)
    b.head_dim, b.page_size = int(head_dim), int(page_size)
    b.sliding_window, b.reserved = int(sliding_window), 0
    b.cu_q_len = _ptr(cu_q_len).value if _ptr(cu_q_len) is not None else None
    b.context_len = _ptr(context_len).value if _ptr(context_len) is not None else None
    b.block_table = _ptr(block_table).value if _ptr(block_table) is not None else None
    return b


def _bf16(t, name):
    if t.dtype != torch.bfloat16 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 tensor")
    return _ptr(t)


def hb_kv_append(batch, k_new, v_new, k_cache, v_cache, stream=None):
    _check(load().hb_kv_append(ctypes.byref(batch), _bf16(k_new, "k_new"),
                               _bf16(v_new, "v_new"), _bf16(k_cache, "k_cache"),
                               _bf16(v_cache, "v_cache"), _stream(stream)))


def hb_plan_sizes(batch, q_len, context_len, num_sms, kv8=False):
    """(plan_bytes, workspace_bytes) for the batch; host-only."""
    ql = np.ascontiguousarray(q_len, dtype=np.int32)
    cl = np.ascontiguousarray(context_len, dtype=np.int32)
    pb, wb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    call = load().hb_kv8_plan if kv8 else load().hb_plan
    _check(call(ctypes.byref(batch), _ptr(ql), _ptr(cl), int(num_sms), None,
                ctypes.byref(pb), None, ctypes.byref(wb), None))
    return pb.value, wb.value


def hb_plan(batch, q_len, context_len, num_sms, workspace=None, stream=None,
            plan=None, upload=True, kv8=False):
    """Write the plan; returns (plan as a host uint8 array, device workspace).

    `workspace` (a uint8 device tensor) is allocated when None or too small.
    With upload=False only the host plan is built (no CUDA call).  kv8: the
    plan of the 8-bit cache's attention (hb_kv8_plan)."""
    call = load().hb_kv8_plan if kv8 else load().hb_plan
    ql = np.ascontiguousarray(q_len, dtype=np.int32)
    cl = np.ascontiguousarray(context_len, dtype=np.int32)
    if plan is not None and (workspace is not None or not upload):
        # buffers given: plan straight into them; ask for sizes only if they
        # turn out too small
        ws = workspace if upload else None
        pb = ctypes.c_size_t(plan.nbytes)
        wb = ctypes.c_size_t(ws.numel() if ws is not None else 0)
        st = call(ctypes.byref(batch), _ptr(ql), _ptr(cl), int(num_sms), _ptr(plan),
                  ctypes.byref(pb), _ptr(ws), ctypes.byref(wb),
                  _stream(stream) if upload else None)
        if st == 0:
            return plan, ws
        if st != 4:   # anything but HB_ERR_WORKSPACE
            _check(st)
    need_p, need_w = hb_plan_sizes(batch, ql, cl, num_sms, kv8)
    if plan is None or plan.nbytes < need_p:
        plan = np.zeros(need_p, dtype=np.uint8)
    if upload and (workspace is None or workspace.numel() < need_w):
        workspace = torch.empty(need_w, dtype=torch.uint8, device="cuda")
    if not upload:
        workspace = None
    pb = ctypes.c_size_t(plan.nbytes)
    wb = ctypes.c_size_t(workspace.numel() if workspace is not None else 0)
    _check(call(ctypes.byref(batch), _ptr(ql), _ptr(cl), int(num_sms),
                _ptr(plan), ctypes.byref(pb), _ptr(workspace),
                ctypes.byref(wb), _stream(stream) if upload else None))
    return plan, workspace


HEADER_BYTES = 176
DECODE_ITEM_INTS = 12
CHUNK_ITEM_INTS = 16


def plan_header(plan):
    """Decode the header of a host plan (for tests and reports)."""
    h = np.frombuffer(plan[:88].tobytes(), dtype=np.int32)
    keys = ("magic", "version", "num_seqs", "total_q", "num_q_heads", "num_kv_heads",
            "head_dim", "page_size", "max_pages_per_seq", "num_sms",
            "num_decode_items", "num_chunk_items", "num_partial_slots",
            "num_merge_counters", "decode_grid", "decode_kvh_block",
            "chunk_tokens_per_tile", "num_chunk_slots", "num_chunk_merges", "sliding_window",
            "num_decode_dynamic", "chunk_pairs_only")
    out = {k: int(v) for k, v in zip(keys, h)}
    u = np.frombuffer(plan[88:HEADER_BYTES].tobytes(), dtype=np.uint64)
    for k, v in zip(("ws_decode_offsets", "items_bytes", "ws_counters", "ws_partial_o",
                     "ws_partial_ml", "ws_total", "plan_bytes", "ws_chunk_counters",
                     "ws_chunk_o", "ws_chunk_ml"), u):
        out[k] = int(v)
    return out


def plan_items(plan):
    """(decode items [n, 12] int32 in interval order, chunk items [m, 16]
    int32, decode interval offsets [grid + num_decode_dynamic + 1]) of a host
    plan: interval b < grid is decode CTA b's static range, the rest are the
    dynamic tail.

    Chunk item columns: seq, kv_head, tok0, ntok, kv_tiles (end), q0, q_len,
    ctx, kv_begin, split, n_splits, slot, merge_id, 3 x padding."""
    hd = plan_header(plan)
    body = plan[HEADER_BYTES:]
    nd, nc = hd["num_decode_items"], hd["num_chunk_items"]
    n_int = nd * DECODE_ITEM_INTS + nc * CHUNK_ITEM_INTS
    ints = np.frombuffer(body[: 4 * n_int].tobytes(), dtype=np.int32)
    dec = ints[: nd * DECODE_ITEM_INTS].reshape(nd, DECODE_ITEM_INTS)
    chk = ints[nd * DECODE_ITEM_INTS: n_int].reshape(nc, CHUNK_ITEM_INTS)
    off = hd["ws_decode_offsets"]
    n_int = hd["decode_grid"] + hd["num_decode_dynamic"]
    offs = np.frombuffer(body[off: off + 4 * (n_int + 1)].tobytes(), dtype=np.int32) \
        if n_int > 0 else np.zeros(1, np.int32)
    return dec, chk, offs


def hb_attention(batch, plan, q, k_cache, v_cache, scale, out, workspace, stream=None):
    _check(load().hb_attention(ctypes.byref(batch), _ptr(plan), _bf16(q, "q"),
                               _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache"),
                               ctypes.c_float(scale), _bf16(out, "out"), _ptr(workspace),
                               _stream(stream)))


def hb_attention_new_kv(batch, plan, q, k_new, v_new, k_cache, v_cache, scale, out, workspace,
                        stream=None):
    """hb_attention that reads the chunks' new K/V rows from k_new / v_new (the
    append's inputs) instead of waiting for the append to write them."""
    _check(load().hb_attention_new_kv(ctypes.byref(batch), _ptr(plan), _bf16(q, "q"),
                                      _bf16(k_new, "k_new"), _bf16(v_new, "v_new"),
                                      _bf16(k_cache, "k_cache"), _bf16(v_cache, "v_cache"),
                                      ctypes.c_float(scale), _bf16(out, "out"), _ptr(workspace),
                                      _stream(stream)))


# ---------------------------------------------------------------- 8-bit cache
# A step makes these calls once per layer, so their checks are one expression
# over everything (about 0.3 us a tensor); only where it fails does _refuse
# look for what to say.
_BF16, _E4M3, _I8, _I32, _I64 = (torch.bfloat16, torch.float8_e4m3fn, torch.int8, torch.int32,
                                 torch.int64)


def _refuse(*specs):
    """Raises for the first (name, tensor, dtype, shape) that does not fit."""
    for name, t, dtype, shape in specs:
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if max(t.shape, default=0) > _INT_MAX:
            raise ValueError(f"{name} has shape {tuple(t.shape)}: over 2^31 - 1")
    for name, t, _, _ in specs:
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device")
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, the current device is "
                             f"cuda:{torch.cuda.current_device()}")
    raise ValueError("arguments on different devices")


def _numel(t):
    return t.numel() if isinstance(t, torch.Tensor) else 0


_INT_MAX = 0x7fffffff      # sizes go to the library as 32-bit integers


def _width(t):
    return t.shape[1] if isinstance(t, torch.Tensor) and t.dim() == 2 else 0


# torch's own short ways to both (0.1 us against 1), where this torch has them;
# called only once a CUDA tensor is at hand
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                       or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))


def _raw_stream(stream, dev):
    if stream is None:
        return _current_raw_stream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def kv8_cache(num_pages, num_kv_heads, head_dim, page_size=16, device="cuda"):
    """A zeroed 8-bit cache: (k_cache, v_cache, k_exp, v_exp)."""
    pools = [torch.zeros(num_pages, page_size, num_kv_heads, head_dim, dtype=torch.uint8,
                         device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    exps = [torch.zeros(num_pages, num_kv_heads, dtype=torch.int8, device=device) for _ in range(2)]
    return (*pools, *exps)


def hb_kv8_append(batch, k_new, v_new, k_cache, v_cache, k_exp, v_exp, stream=None):
    """Quantise the batch's new K/V rows (bf16) into the 8-bit cache."""
    pages, hkv, d = batch.num_pages, batch.num_kv_heads, batch.head_dim
    new, pool, exps = (batch.total_q, hkv, d), (pages, batch.page_size, hkv, d), (pages, hkv)
    try:
        dev = k_new.get_device()
        ok = (k_new.dtype is _BF16 and k_new.shape == new and k_new.is_contiguous()
              and v_new.dtype is _BF16 and v_new.shape == new and v_new.is_contiguous()
              and k_cache.dtype is _E4M3 and k_cache.shape == pool and k_cache.is_contiguous()
              and v_cache.dtype is _E4M3 and v_cache.shape == pool and v_cache.is_contiguous()
              and k_exp.dtype is _I8 and k_exp.shape == exps and k_exp.is_contiguous()
              and v_exp.dtype is _I8 and v_exp.shape == exps and v_exp.is_contiguous()
              and dev >= 0 and dev == v_new.get_device() == k_cache.get_device()
              == v_cache.get_device() == k_exp.get_device() == v_exp.get_device()
              and dev == _current_device())
    except AttributeError:
        ok = False
    if not ok:
        _refuse(("k_new", k_new, _BF16, new), ("v_new", v_new, _BF16, new),
                ("k_cache", k_cache, _E4M3, pool), ("v_cache", v_cache, _E4M3, pool),
                ("k_exp", k_exp, _I8, exps), ("v_exp", v_exp, _I8, exps))
    st = (_lib or load()).hb_kv8_append(
        ctypes.byref(batch), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), _raw_stream(stream, dev))
    if st:
        _check(st)


def hb_kv8_plan(batch, q_len, context_len, num_sms, workspace=None, stream=None, plan=None,
                upload=True):
    """hb_plan for hb_kv8_attention."""
    return hb_plan(batch, q_len, context_len, num_sms, workspace, stream, plan, upload, kv8=True)


_CHAR = ctypes.c_char
_PLAN_SIZES = struct.Struct("<QQ")       # plan_header()["ws_total"], ["plan_bytes"]
_PLAN_SIZES_AT = 88 + 8 * 5


def hb_kv8_attention(batch, plan, q, k_cache, v_cache, k_exp, v_exp, scale, out, workspace,
                     stream=None):
    """hb_attention over the 8-bit cache."""
    pages, hkv, d = batch.num_pages, batch.num_kv_heads, batch.head_dim
    rows, pool, exps = (batch.total_q, batch.num_q_heads, d), (pages, batch.page_size, hkv, d), (pages, hkv)
    if (not isinstance(plan, np.ndarray) or plan.dtype != np.uint8 or plan.nbytes < HEADER_BYTES
            or not plan.flags.c_contiguous):
        raise ValueError("plan must be the uint8 array that hb_kv8_plan returned")
    need, size = _PLAN_SIZES.unpack_from(plan, _PLAN_SIZES_AT)
    if plan.nbytes < size:   # (the library reads it at places that the header gives)
        raise ValueError(f"plan has {plan.nbytes} bytes of the {size} that hb_kv8_plan wrote")
    have = _numel(workspace) if workspace is not None else need
    if have < need:
        raise ValueError(f"workspace has {have} bytes, the plan needs {need}")
    try:
        dev = q.get_device()
        ok = (q.dtype is _BF16 and q.shape == rows and q.is_contiguous()
              and out.dtype is _BF16 and out.shape == rows and out.is_contiguous()
              and k_cache.dtype is _E4M3 and k_cache.shape == pool and k_cache.is_contiguous()
              and v_cache.dtype is _E4M3 and v_cache.shape == pool and v_cache.is_contiguous()
              and k_exp.dtype is _I8 and k_exp.shape == exps and k_exp.is_contiguous()
              and v_exp.dtype is _I8 and v_exp.shape == exps and v_exp.is_contiguous()
              and dev >= 0 and dev == out.get_device() == k_cache.get_device()
              == v_cache.get_device() == k_exp.get_device() == v_exp.get_device()
              and dev == _current_device()
              and (workspace is None or (workspace.dtype is torch.uint8 and workspace.dim() == 1
                                         and workspace.is_contiguous()
                                         and workspace.get_device() == dev)))
    except AttributeError:
        ok = False
    if not ok:
        specs = [("q", q, _BF16, rows), ("k_cache", k_cache, _E4M3, pool),
                 ("v_cache", v_cache, _E4M3, pool), ("k_exp", k_exp, _I8, exps),
                 ("v_exp", v_exp, _I8, exps), ("out", out, _BF16, rows)]
        if workspace is not None:
            specs.append(("workspace", workspace, torch.uint8, (have,)))
        _refuse(*specs)
    try:
        at = ctypes.byref(_CHAR.from_buffer(plan))   # (0.3 us; plan.ctypes.data 0.9)
    except TypeError:                                # (read-only)
        at = plan.ctypes.data
    st = (_lib or load()).hb_kv8_attention(
        ctypes.byref(batch), at, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        k_exp.data_ptr(), v_exp.data_ptr(), scale, out.data_ptr(),
        workspace.data_ptr() if workspace is not None else None, _raw_stream(stream, dev))
    if st:
        _check(st)


# ---------------------------------------------------------------- pages on the GPU
def pages_ring(num_pages, page_order=None, device="cuda"):
    """A ring with every page free: (free_pages, state) for hb_pages_*."""
    ring = torch.arange(num_pages, dtype=torch.int32) if page_order is None else \
        torch.as_tensor(page_order, dtype=torch.int32)
    if ring.dim() != 1 or not torch.equal(ring.sort().values.cpu(), torch.arange(num_pages, dtype=torch.int32)):
        raise ValueError("page_order must list every page once")
    return ring.to(device), torch.tensor([0, num_pages, 0, 0], dtype=torch.int64, device=device)


def hb_pages_assign(q_len, context_len, free_pages, state_in, state_out, block_table, cu_q_len,
                    slot_map=None, page_size=16, stream=None):
    """Block-table entries, prefix sums and (if given) slots of a step from its
    lengths on the GPU, with pages taken from the ring free_pages / state_in
    (state_out receives the ring's new state and may be state_in)."""
    state = (4,)
    try:
        n, pages = q_len.numel(), free_pages.numel()
        max_pages = block_table.shape[1] if block_table.dim() == 2 else 0
        slots = min(slot_map.numel(), _INT_MAX) if slot_map is not None else _INT_MAX
        rows, table = (n,), (n, max_pages)
        dev = q_len.get_device()
        ok = (pages <= _INT_MAX and max_pages <= _INT_MAX and n <= _INT_MAX
              and q_len.dtype is _I32 and q_len.shape == rows and q_len.is_contiguous()
              and context_len.dtype is _I32 and context_len.shape == rows and context_len.is_contiguous()
              and free_pages.dtype is _I32 and free_pages.dim() == 1 and free_pages.is_contiguous()
              and state_in.dtype is _I64 and state_in.shape == state and state_in.is_contiguous()
              and state_out.dtype is _I64 and state_out.shape == state and state_out.is_contiguous()
              and block_table.dtype is _I32 and block_table.shape == table
              and block_table.is_contiguous()
              and cu_q_len.dtype is _I32 and cu_q_len.shape == (n + 1,) and cu_q_len.is_contiguous()
              and dev >= 0 and dev == context_len.get_device() == free_pages.get_device()
              == state_in.get_device() == state_out.get_device() == block_table.get_device()
              == cu_q_len.get_device() and dev == _current_device()
              and (slot_map is None or (slot_map.dtype is _I64 and slot_map.dim() == 1
                                        and slot_map.is_contiguous()
                                        and slot_map.get_device() == dev)))
    except AttributeError:
        ok = False
    if not ok:
        n = _numel(q_len)
        specs = [("q_len", q_len, _I32, (n,)), ("context_len", context_len, _I32, (n,)),
                 ("free_pages", free_pages, _I32, (_numel(free_pages),)),
                 ("state_in", state_in, _I64, state), ("state_out", state_out, _I64, state),
                 ("block_table", block_table, _I32, (n, _width(block_table))),
                 ("cu_q_len", cu_q_len, _I32, (n + 1,))]
        if slot_map is not None:
            specs.append(("slot_map", slot_map, _I64, (_numel(slot_map),)))
        _refuse(*specs)
    st = (_lib or load()).hb_pages_assign(
        n, slots, max_pages, pages, page_size, q_len.data_ptr(), context_len.data_ptr(),
        free_pages.data_ptr(), state_in.data_ptr(), state_out.data_ptr(), block_table.data_ptr(),
        cu_q_len.data_ptr(), slot_map.data_ptr() if slot_map is not None else None,
        _raw_stream(stream, dev))
    if st:
        _check(st)


def hb_pages_release(lengths, free_pages, state_in, state_out, block_table, page_size=16,
                     stream=None):
    """The pages of the sequences with lengths > 0 (tokens in the cache) go back
    to the ring."""
    state = (4,)
    try:
        n, pages = lengths.numel(), free_pages.numel()
        max_pages = block_table.shape[1] if block_table.dim() == 2 else 0
        rows, table = (n,), (n, max_pages)
        dev = lengths.get_device()
        ok = (pages <= _INT_MAX and max_pages <= _INT_MAX and n <= _INT_MAX
              and lengths.dtype is _I32 and lengths.shape == rows and lengths.is_contiguous()
              and block_table.dtype is _I32 and block_table.shape == table
              and block_table.is_contiguous()
              and free_pages.dtype is _I32 and free_pages.dim() == 1 and free_pages.is_contiguous()
              and state_in.dtype is _I64 and state_in.shape == state and state_in.is_contiguous()
              and state_out.dtype is _I64 and state_out.shape == state and state_out.is_contiguous()
              and dev >= 0 and dev == block_table.get_device() == free_pages.get_device()
              == state_in.get_device() == state_out.get_device() and dev == _current_device())
    except AttributeError:
        ok = False
    if not ok:
        n = _numel(lengths)
        _refuse(("lengths", lengths, _I32, (n,)),
                ("block_table", block_table, _I32, (n, _width(block_table))),
                ("free_pages", free_pages, _I32, (_numel(free_pages),)),
                ("state_in", state_in, _I64, state), ("state_out", state_out, _I64, state))
    st = (_lib or load()).hb_pages_release(
        n, max_pages, pages, page_size, lengths.data_ptr(), block_table.data_ptr(),
        free_pages.data_ptr(), state_in.data_ptr(), state_out.data_ptr(), _raw_stream(stream, dev))
    if st:
        _check(st)


def hb_decode_attention_noalloc(batch, q_len, context_len, q, k_cache, v_cache, scale,
                                out, stream=None):
    """Decode-row attention with the library's static scratch (no workspace,
    no device allocation by the library); all rows must have q_len == 1."""
    ql = np.ascontiguousarray(q_len, dtype=np.int32)
    cl = np.ascontiguousarray(context_len, dtype=np.int32)
    _check(load().hb_decode_attention_noalloc(
        ctypes.byref(batch), _ptr(ql), _ptr(cl), _bf16(q, "q"), _bf16(k_cache, "k_cache"),
        _bf16(v_cache, "v_cache"), ctypes.c_float(scale), _bf16(out, "out"),
        _stream(stream)))


def hb_check(stream=None):
    _check(load().hb_check(_stream(stream)))


def hb_selftest_wait_timeout(stream=None):
    _check(load().hb_selftest_wait_timeout(_stream(stream)))


def hb_selftest_flag_timeout(stream=None):
    _check(load().hb_selftest_flag_timeout(_stream(stream)))


def hb_timing_enable(on: bool, keep: bool = False):
    """Start (clearing earlier records; with keep=True resuming) or stop
    recording launch durations."""
    _check(load().hb_timing_enable((2 if keep else 1) if on else 0))


def hb_timing_read():
    """{kernel name: (total ms, launches)} since timing was enabled."""
    ms = (ctypes.c_double * HB_NUM_KERNEL_IDS)()
    n = (ctypes.c_int32 * HB_NUM_KERNEL_IDS)()
    _check(load().hb_timing_read(ms, n))
    return {KERNEL_NAMES[i]: (ms[i], n[i]) for i in range(HB_NUM_KERNEL_IDS)}


def hb_timing_durations(kernel):
    """Per-launch durations (ms, launch order) recorded for one kernel name."""
    k = KERNEL_NAMES.index(kernel)
    n = ctypes.c_int32(0)
    _check(load().hb_timing_durations(k, None, 0, ctypes.byref(n)))
    buf = (ctypes.c_float * max(1, n.value))()
    _check(load().hb_timing_durations(k, buf, n.value, ctypes.byref(n)))
    return [float(buf[i]) for i in range(n.value)]


def hb_step_layout(batch):
    """(section offsets [q, k_new, v_new, cu_q_len, context_len, block_table],
    total bytes) of hb_step's packed input block for this batch's sizes."""
    offs = (ctypes.c_size_t * HB_STEP_SECTIONS)()
    n = ctypes.c_size_t(0)
    _check(load().hb_step_layout(ctypes.byref(batch), offs, ctypes.byref(n)))
    return list(offs), n.value


class StepSlot:
    """hb_step_slot: the events that order one set of staging buffers' copies
    and kernels (created on the current device)."""

    def __init__(self):
        h = ctypes.c_void_p()
        _check(load().hb_step_slot_create(ctypes.byref(h)))
        self._h = h

    def sync(self):
        _check(load().hb_step_slot_sync(self._h))

    def close(self):
        if self._h:
            load().hb_step_slot_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def hb_step(batch, q_len, context_len, num_sms, slot, buffers, k_cache, v_cache, scale,
            copy_in_stream, stream, copy_out_stream):
    """One step from host memory (see hb.h).  `buffers` is an HbStepBuffers;
    q_len / context_len are host int32 arrays (kept contiguous by the
    caller for repeated calls)."""
    _check(load().hb_step(ctypes.byref(batch), _ptr(q_len), _ptr(context_len), int(num_sms),
                          slot._h, ctypes.byref(buffers), _bf16(k_cache, "k_cache"),
                          _bf16(v_cache, "v_cache"), ctypes.c_float(scale),
                          _stream(copy_in_stream), _stream(stream), _stream(copy_out_stream)))


def hb_launch_count() -> int:
    return int(load().hb_launch_count())


class Builder:
    """The library's stall-free batch builder (host only)."""

    def __init__(self, budget, page_size, num_pages, max_pages_per_seq, page_order=None):
        self.max_pages_per_seq = max_pages_per_seq
        handle = ctypes.c_void_p()
        order = None
        if page_order is not None:
            order = np.ascontiguousarray(page_order, dtype=np.int32)
        _check(load().hb_builder_create(budget, page_size, num_pages, max_pages_per_seq,
                                        _ptr(order), ctypes.byref(handle)), builder=True)
        self._h = handle
        self._max_rows = 64

    def close(self):
        if self._h:
            load().hb_builder_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_request(self, rid, prompt_len, max_new):
        _check(load().hb_builder_add_request(self._h, int(rid), int(prompt_len),
                                             int(max_new)), builder=True)

    def step(self):
        """Next batch as a dict of numpy arrays, or None when there is nothing to run."""
        while True:
            mr, mp = self._max_rows, self.max_pages_per_seq
            # the library writes every entry of the rows it returns (block
            # table entries past a row's pages as -1); the rest is not read
            ql = np.empty(mr, np.int32)
            cl = np.empty(mr, np.int32)
            bt = np.empty((mr, mp), np.int32)
            ids = np.empty(mr, np.int64)
            kind = np.empty(mr, np.int32)
            n, over = ctypes.c_int32(0), ctypes.c_int32(0)
            st = load().hb_builder_step(self._h, mr, ctypes.byref(n), _ptr(ql), _ptr(cl),
                                        _ptr(bt), _ptr(ids), _ptr(kind), ctypes.byref(over))
            if st == 4 and n.value > mr:      # HB_ERR_WORKSPACE: grow and retry
                self._max_rows = n.value
                continue
            _check(st, builder=True)
            k = n.value
            if k == 0:
                return None
            return {"q_len": ql[:k], "context_len": cl[:k], "block_table": bt[:k],
                    "ids": ids[:k], "kind": kind[:k], "over_budget": bool(over.value)}

    def complete(self):
        out = np.zeros(max(self._max_rows, 1), np.int64)
        n = ctypes.c_int32(0)
        _check(load().hb_builder_complete(self._h, out.size, ctypes.byref(n), _ptr(out)),
               builder=True)
        return [int(x) for x in out[: n.value]]

    def counts(self):
        w, r, f = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(load().hb_builder_counts(self._h, ctypes.byref(w), ctypes.byref(r),
                                        ctypes.byref(f)), builder=True)
        return w.value, r.value, f.value

    def free_list(self):
        _, _, nfree = self.counts()
        out = np.zeros(max(nfree, 1), np.int32)
        n = ctypes.c_int32(0)
        _check(load().hb_builder_free_list(self._h, out.size, ctypes.byref(n), _ptr(out)),
               builder=True)
        return [int(x) for x in out[: n.value]]


_linear_ws = {}


def linear_workspace(M, N, K, epilogue, device=None):
    """A zero-filled device workspace big enough for hb_linear's split-K on
    this problem (cached per device and grown as needed), or None."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    need = int(load().hb_linear_workspace_size(int(M), int(N), int(K), int(epilogue), sms))
    if need == 0:
        return None
    ws = _linear_ws.get(dev)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, dtype=torch.uint8, device=dev)
        _linear_ws[dev] = ws
    return ws


def hb_linear(x, w, outs, epilogue=LINEAR_STORE, stream=None, workspace="auto"):
    """y = x w^T on the tensor cores.  x [M, K], w [N, K] bf16 device tensors;
    outs: the destination tensors ([M, cols_i] bf16 each; their column
    counts split N for STORE / RESIDUAL, one [M, N / 2] tensor for GATED).
    workspace: "auto" (a cached zero-filled device buffer for split-K when
    the problem has few tiles), None (no split), or a uint8 device tensor."""
    if len(outs) > 3:
        raise ValueError("at most three destinations")
    o = HbLinearOut()
    for i, t in enumerate(outs):
        _bf16(t, "out")
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError("each destination must be a contiguous 2-D tensor")
        o.y[i] = t.data_ptr()
        o.cols[i] = t.shape[1]
    M, N, K = int(x.shape[0]), int(w.shape[0]), int(x.shape[1])
    if isinstance(workspace, str):
        workspace = linear_workspace(M, N, K, epilogue, x.device) if M > 0 else None
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().hb_linear(_bf16(x, "x"), _bf16(w, "w"), M, N, K, int(epilogue),
                            ctypes.byref(o), ws_ptr, ws_bytes, _stream(stream)))


# ---------------------------------------------------------------- norms
_F32 = torch.float32
_NORM_ARGS = struct.Struct("<4i7Q5q4f")     # HbNormArgs
assert _NORM_ARGS.size == ctypes.sizeof(HbNormArgs)


def _refuse_rows(*specs):
    """Raises for the first (name, tensor, dtypes, shape) that does not fit, or
    whose rows (the last dimensions) are not dense."""
    for name, t, dtypes, shape in specs:
        if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
            raise ValueError(f"{name} must be a {' or '.join(str(d) for d in dtypes)} tensor")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if max(t.shape, default=0) > _INT_MAX:
            raise ValueError(f"{name} has shape {tuple(t.shape)}: over 2^31 - 1")
        if t.numel() and not t[0].is_contiguous():
            raise ValueError(f"{name}: each row must be contiguous")
    for name, t, _, _ in specs:
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device")
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, the current device is "
                             f"cuda:{torch.cuda.current_device()}")


def hb_norm(x=None, y=None, x_out=None, z=None, w_pre=None, w_post=None, gate=None, eps=1e-6, residual_scale=1.0,
            branch_scale=1.0, weight_offset=0.0, stream=None):
    """The norm after a branch (w_post), its gate, the residual sum and the norm
    before the next branch, over [rows, width] tensors (rows may be apart):

        u     = norm(y, w_post), or y
        x_out = residual_scale * x + branch_scale * gate * u
        z     = norm(x_out, w_pre)

    y, z and the weights are bf16, x and x_out both bf16 or both fp32, gate
    [width] or [rows, width] (or [1, width]) bf16.  What is None drops out; x_out
    and z may be x or y (in place)."""
    lead = x if x is not None else y
    if not isinstance(lead, torch.Tensor) or lead.dim() != 2:
        raise ValueError("x or y must be a [rows, width] tensor")
    shape, dev = lead.shape, lead.get_device()
    rows, width = shape
    kind = x.dtype if x is not None else (x_out.dtype if isinstance(x_out, torch.Tensor) else _BF16)
    # (addresses and strides of what is given; the struct's fields set one by one take twice as long)
    px = py = pg = pp = pw = po = pz = sx = sy = sg = so = sz = 0
    try:
        ok = ((kind is _BF16 or kind is _F32) and rows <= _INT_MAX and 0 < width <= _INT_MAX and dev >= 0
              and dev == _current_device())
        if x is not None:
            sx, one = x.stride()
            ok, px = ok and one == 1, x.data_ptr()
        if y is not None:
            sy, one = y.stride()
            ok = ok and one == 1 and y.dtype is _BF16 and y.shape == shape and y.get_device() == dev
            py = y.data_ptr()
        if x_out is not None:
            so, one = x_out.stride()
            ok = ok and one == 1 and x_out.dtype is kind and x_out.shape == shape and x_out.get_device() == dev
            po = x_out.data_ptr()
        if z is not None:
            sz, one = z.stride()
            ok = ok and one == 1 and z.dtype is _BF16 and z.shape == shape and z.get_device() == dev
            pz = z.data_ptr()
        if w_pre is not None:
            ok = (ok and w_pre.dtype is _BF16 and w_pre.shape == (width,) and w_pre.is_contiguous()
                  and w_pre.get_device() == dev)
            pw = w_pre.data_ptr()
        if w_post is not None:
            ok = (ok and w_post.dtype is _BF16 and w_post.shape == (width,) and w_post.is_contiguous()
                  and w_post.get_device() == dev)
            pp = w_post.data_ptr()
        if gate is not None:
            each = gate.dim() == 2 and gate.shape[0] == rows and rows > 1
            ok = (ok and gate.dtype is _BF16 and (each or gate.numel() == width) and gate.shape[-1] == width
                  and gate.stride(-1) == 1 and gate.get_device() == dev)
            pg, sg = gate.data_ptr(), gate.stride(0) if each else 0
    except (AttributeError, IndexError, ValueError):
        ok = False
    if not ok:
        stream_t = (kind if kind in (_BF16, _F32) else _BF16,)
        specs = [("x", x, (_BF16, _F32), shape), ("y", y, (_BF16,), shape), ("x_out", x_out, stream_t, shape),
                 ("z", z, (_BF16,), shape), ("w_pre", w_pre, (_BF16,), (width,)),
                 ("w_post", w_post, (_BF16,), (width,))]
        if gate is not None:
            each = isinstance(gate, torch.Tensor) and gate.dim() == 2
            specs.append(("gate", gate, (_BF16,), ((1 if _numel(gate) == width else rows), width) if each else (width,)))
        _refuse_rows(*(s for s in specs if s[1] is not None))
        raise ValueError("width must be > 0, and the tensors on one device")
    if rows == 0:
        return
    st = (_lib or load()).hb_norm(
        _NORM_ARGS.pack(rows, width, 1 if kind is _F32 else 0, 0, px, py, pg, pp, pw, po, pz, sx, sy, sg, so, sz, eps,
                        residual_scale, branch_scale, weight_offset), _raw_stream(stream, dev))
    if st:
        _check(st)


# ---------------------------------------------------------------- rotary positions
def rope_phases(rotary_dim, base=10000.0, scaling="none", scale_by=1.0, original_context=0, parts=(1.0, 32.0)):
    """What each pair of a head turns by from one position to the next, in
    2^-64 of a turn (a host uint64 array; see hb_rope_phases)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALINGS)}")
    out = np.zeros(max(0, int(rotary_dim)) // 2, np.uint64)
    _check(load().hb_rope_phases(int(rotary_dim), base, ROPE_SCALINGS.index(scaling), scale_by, original_context,
                                 parts[0], parts[1], out.ctypes.data))
    return out


def make_rope(rotary_dim, base=10000.0, scaling="none", scale_by=1.0, original_context=0, parts=(1.0, 32.0),
              interleaved=False, factor=1.0, q_weight=None, k_weight=None, eps=1e-6, device="cuda") -> HbRopeParams:
    """hb_rope's parameters, with the phases on the device.  rotary_dim 0: head
    norms alone.  scaling "parts" goes by the turns that a pair makes over
    original_context, linearly between the two of `parts`; ramps over the pair
    index and factors per pair are other tables, which this does not make.  Made
    once per model; the tensors live as long as it."""
    r = HbRopeParams()
    r.rotary_dim, r.interleaved, r.factor, r.eps = int(rotary_dim), int(bool(interleaved)), factor, eps
    keep = []
    if r.rotary_dim:
        phases = torch.from_numpy(rope_phases(rotary_dim, base, scaling, scale_by, original_context,
                                              parts).view(np.int64)).to(device)
        keep.append(phases)
        r.phases = phases.data_ptr()
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            if w.dtype != torch.bfloat16 or w.dim() != 1 or not w.is_contiguous():
                raise ValueError(f"{name} must be a contiguous [head_dim] bfloat16 tensor")
            if w.device.type != torch.device(device).type:
                raise ValueError(f"{name} is on {w.device}, not on {device}")
            if keep and w.get_device() != keep[0].get_device():
                raise ValueError(f"{name} is on {w.device}, not on {keep[0].device}")
            keep.append(w)
            setattr(r, name, w.data_ptr())
    r.tensors, r.head_dims = tuple(keep), {w.numel() for w in (q_weight, k_weight) if w is not None}
    r.device_index = keep[0].get_device() if keep else None
    return r


def _token_stride(t, row):
    """Elements between tokens whose heads (of `row` elements) stand one behind the
    other; -1 where they do not.  (A stride costs three times what is_contiguous does.)"""
    if t.is_contiguous():
        return row
    first, head, one = t.stride()
    return first if one == 1 and (head == t.shape[2] or t.shape[1] == 1) else -1


def _in_place_or_dense(out, source, row):
    """out: source itself, or contiguous (and not at its place with another stride)."""
    if out is source:
        return True
    if out.data_ptr() != source.data_ptr():
        return out.is_contiguous()
    return out.shape[0] == 1 or _token_stride(out, row) == _token_stride(source, row) >= 0


def hb_rope(batch, rope, q, k, v, q_out, k_out, k_cache, v_cache, stream=None):
    """Rotary positions of the batch's q [total_q, Hq, D] and k [total_q, Hkv, D]
    (after head norms where `rope` has weights), with k and v put into their cache
    pages.  q, k and v may be columns of one tensor (dense heads, tokens a stride
    apart); q_out and k_out are q and k themselves or contiguous tensors; k_out
    may be None; v, k_cache and v_cache are all None where nothing is to be
    appended."""
    hq, hkv, d, n = batch.num_q_heads, batch.num_kv_heads, batch.head_dim, batch.total_q
    q_rows, k_rows, pool = (n, hq, d), (n, hkv, d), (batch.num_pages, batch.page_size, hkv, d)
    q_row, k_row, v_stride = hq * d, hkv * d, 0
    try:
        dev = q.get_device()
        q_stride, k_stride = _token_stride(q, q_row), _token_stride(k, k_row)
        ok = (q.dtype is _BF16 and q.shape == q_rows and q_stride >= 0
              and k.dtype is _BF16 and k.shape == k_rows and k_stride >= 0
              and q_out.dtype is _BF16 and q_out.shape == q_rows and _in_place_or_dense(q_out, q, q_row)
              and dev >= 0 and dev == k.get_device() == q_out.get_device() and dev == _current_device()
              and (rope.device_index is None or rope.device_index == dev)
              and (not rope.head_dims or rope.head_dims == {d}))
        if k_out is not None:
            ok = (ok and k_out.dtype is _BF16 and k_out.shape == k_rows and k_out.get_device() == dev
                  and _in_place_or_dense(k_out, k, k_row))
        if k_cache is not None:
            v_stride = _token_stride(v, k_row)
            ok = (ok and v.dtype is _BF16 and v.shape == k_rows and v_stride >= 0 and v.get_device() == dev
                  and k_cache.dtype is _BF16 and k_cache.shape == pool and k_cache.is_contiguous()
                  and v_cache.dtype is _BF16 and v_cache.shape == pool and v_cache.is_contiguous()
                  and k_cache.get_device() == dev == v_cache.get_device())
        else:
            ok = ok and v is None and v_cache is None
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _refuse_rope(rope, d, (("q", q, q_rows), ("k", k, k_rows), ("v", v, k_rows)),
                     (("q_out", q_out, q_rows, q), ("k_out", k_out, k_rows, k)),
                     (("k_cache", k_cache, pool), ("v_cache", v_cache, pool)))
    if n == 0:
        return
    # (data_ptr() of an empty pool is 0; the library refuses it)
    st = (_lib or load()).hb_rope(
        ctypes.byref(batch), ctypes.byref(rope), q.data_ptr(), q_stride, k.data_ptr(), k_stride,
        v.data_ptr() if v is not None else None, v_stride, q_out.data_ptr(),
        k_out.data_ptr() if k_out is not None else None, k_cache.data_ptr() if k_cache is not None else None,
        v_cache.data_ptr() if v_cache is not None else None, _raw_stream(stream, dev))
    if st:
        _check(st)


def _refuse_rope(rope, d, ins, outs, pools):
    if not isinstance(rope, HbRopeParams) or not hasattr(rope, "tensors"):
        raise ValueError("rope must be what make_rope returned")
    if rope.head_dims and rope.head_dims != {d}:
        raise ValueError(f"the head norms' weights have {sorted(rope.head_dims)} elements, head_dim is {d}")
    cached = [x is not None for x in (ins[2][1], pools[0][1], pools[1][1])]
    if any(cached) != all(cached):
        raise ValueError("v, k_cache and v_cache go together")
    if not all(isinstance(x[1], torch.Tensor) for x in ins[:2]):
        raise ValueError("q and k must be tensors")
    specs = [(name, t, (_BF16,), shape) for name, t, shape in ins if t is not None or name != "v"]
    specs += [(name, t, (_BF16,), shape) for name, t, shape, _ in outs if t is not None or name != "k_out"]
    specs += [(name, t, (_BF16,), shape) for name, t, shape in pools if t is not None]
    for name, t, _, _ in specs:
        if isinstance(t, torch.Tensor) and name.endswith("cache") and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for name, t, shape, source in outs:
        if (isinstance(t, torch.Tensor) and isinstance(source, torch.Tensor) and t.dim() == 3 and source.dim() == 3
                and not _in_place_or_dense(t, source, t.shape[1] * t.shape[2])):
            raise ValueError(f"{name} must be contiguous, or {name[0]} itself")
    _refuse_rows(*specs)
    if rope.device_index is not None and rope.device_index != torch.cuda.current_device():
        raise ValueError(f"rope's tensors are on cuda:{rope.device_index}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    raise ValueError("q, k and v: heads must be dense, and all tensors on one device")


# ---------------------------------------------------------------- low-rank adapters
def make_adapters(a, b, rank, scale, cols) -> HbAdapterPool:
    """The pool of one projection's adapters: a [n, len(cols), max_rank, K] and b
    [n, sum(cols), max_rank] bf16, rank [n] int32 and scale [n] fp32 on the device
    (they may be written into, to bring adapters in and out; they live as long as
    the pool); cols: the columns of the projection's destinations."""
    cols = tuple(int(c) for c in cols)
    if not 1 <= len(cols) <= 3 or min(cols) <= 0:
        raise ValueError("cols must be one to three positive column counts")
    if not isinstance(a, torch.Tensor) or a.dim() != 4 or a.shape[0] == 0:
        raise ValueError("a must be a [num_adapters, destinations, max_rank, K] tensor")
    n, _, r, k = a.shape
    for name, t, dtype, shape in (("a", a, _BF16, (n, len(cols), r, k)), ("b", b, _BF16, (n, sum(cols), r)),
                                  ("rank", rank, _I32, (n,)), ("scale", scale, _F32, (n,))):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor")
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        if max(t.shape) > _INT_MAX:
            raise ValueError(f"{name} has shape {tuple(t.shape)}: over 2^31 - 1")
        if t.device != a.device:
            raise ValueError(f"{name} is on {t.device}, a on {a.device}")
    p = HbAdapterPool()
    p.num_adapters, p.max_rank, p.K, p.N, p.slices = n, r, k, sum(cols), len(cols)
    p.a, p.b, p.rank, p.scale = a.data_ptr(), b.data_ptr(), rank.data_ptr(), scale.data_ptr()
    p.tensors, p.cols, p.device_index = (a, b, rank, scale), cols, a.get_device()
    return p


_ADAPTER_PLAN_BYTES = 88
_ADAPTER_PLAN_INTS = struct.Struct("<I11i")
_ADAPTER_PLAN_SIZES = struct.Struct("<QQ")      # workspace, plan
_ADAPTER_PLAN_SIZES_AT = 48 + 3 * 8
_LINEAR_OUT = struct.Struct("<3Q3i4x")          # HbLinearOut
assert _LINEAR_OUT.size == ctypes.sizeof(HbLinearOut)


def adapters_plan_header(plan):
    """The header of an adapter plan (for tests and reports)."""
    keys = ("magic", "num_seqs", "total_q", "num_adapters", "max_ranks", "num_sms", "num_long", "num_short",
            "num_idle", "long_rows", "short_rows", "short_pieces")
    out = dict(zip(keys, _ADAPTER_PLAN_INTS.unpack_from(plan)))
    out["ws_total"], out["plan_bytes"] = _ADAPTER_PLAN_SIZES.unpack_from(plan, _ADAPTER_PLAN_SIZES_AT)
    return out


def adapters_plan_items(plan):
    """(segments [n, 4]: adapter, first entry of the row list, rows, first token of a
    long tile or -1; row list) of an adapter plan."""
    h = adapters_plan_header(plan)
    n = h["num_long"] + h["num_short"] + h["num_idle"]
    body = plan[_ADAPTER_PLAN_BYTES:h["plan_bytes"]].tobytes()
    return np.frombuffer(body[:16 * n], np.int32).reshape(n, 4), np.frombuffer(body[16 * n:], np.int32)


def _host_int32(name, values):
    """A host array of whole numbers as int32; those that do not fit are refused, not cut."""
    a = np.asarray(values)
    if a.size and (a.dtype.kind not in "iu" or int(a.min()) < -_INT_MAX - 1 or int(a.max()) > _INT_MAX):
        raise ValueError(f"{name} must be whole numbers of 32 bits")
    return np.ascontiguousarray(a, dtype=np.int32)


def hb_adapters_plan(pools, q_len, adapter, num_sms, total_q=None, workspace=None, plan=None, stream=None, upload=True):
    """Sort a batch's tokens by adapter: q_len and each sequence's adapter (-1: none),
    host arrays.  `pools`: a pool or several (the step's projections) of as many
    adapters.  Returns (plan as a host uint8 array, device workspace), for
    hb_adapters with any of them; as hb_plan."""
    pools = (pools,) if isinstance(pools, HbAdapterPool) else tuple(pools)
    if not pools or any(p.num_adapters != pools[0].num_adapters for p in pools):
        raise ValueError("the pools of a plan have as many adapters")
    ql, of = _host_int32("q_len", q_len), _host_int32("adapter", adapter)
    if ql.ndim != 1 or ql.shape != of.shape:
        raise ValueError(f"q_len has shape {ql.shape}, adapter {of.shape}")
    total = int(ql.sum(dtype=np.int64)) if total_q is None else int(total_q)
    if total > _INT_MAX:
        raise ValueError(f"{total} tokens: over 2^31 - 1")
    ranks = max(p.slices * p.max_rank for p in pools)

    def call(plan, workspace):
        pb = ctypes.c_size_t(plan.nbytes if plan is not None else 0)
        wb = ctypes.c_size_t(workspace.numel() if workspace is not None else 0)
        return load().hb_adapters_plan(
            len(ql), total, _ptr(ql), _ptr(of), pools[0].num_adapters, ranks, int(num_sms), _ptr(plan),
            ctypes.byref(pb), _ptr(workspace), ctypes.byref(wb), _stream(stream) if workspace is not None else None), \
            pb.value, wb.value
    if plan is not None and (workspace is not None or not upload):
        st, _, _ = call(plan, workspace if upload else None)
        if st == 0:
            return plan, workspace if upload else None
        if st != 4:   # anything but HB_ERR_WORKSPACE
            _check(st)
    st, need_p, need_w = call(None, None)
    _check(st)
    if plan is None or plan.nbytes < need_p:
        plan = np.zeros(need_p, dtype=np.uint8)
    if not upload:
        workspace = None
    elif workspace is None or workspace.numel() < need_w:
        workspace = torch.empty(max(need_w, 256), dtype=torch.uint8, device="cuda")
    _check(call(plan, workspace)[0])
    return plan, workspace


def hb_adapters(pool, plan, x, y, out, workspace, stream=None):
    """out_i = y_i + scale (x A_i^T) B_i^T with each token's own adapter: x [total_q,
    K], y and out lists of [total_q, cols_i] tensors (out may be y: in place)."""
    if (not isinstance(plan, np.ndarray) or plan.dtype != np.uint8 or plan.nbytes < _ADAPTER_PLAN_BYTES
            or not plan.flags.c_contiguous):
        raise ValueError("plan must be the uint8 array that hb_adapters_plan returned")
    need, size = _ADAPTER_PLAN_SIZES.unpack_from(plan, _ADAPTER_PLAN_SIZES_AT)
    if plan.nbytes < size:
        raise ValueError(f"plan has {plan.nbytes} bytes of the {size} that hb_adapters_plan wrote")
    if not isinstance(pool, HbAdapterPool) or not hasattr(pool, "cols"):
        raise ValueError("pool must be what make_adapters returned")
    rows, cols = _ADAPTER_PLAN_INTS.unpack_from(plan)[2], pool.cols
    src, dst = [], []
    try:
        dev = x.get_device()
        ok = (x.dtype is _BF16 and x.shape == (rows, pool.K) and x.is_contiguous() and dev >= 0
              and dev == pool.device_index and dev == _current_device() and len(y) == len(out) == len(cols)
              and workspace.dtype is torch.uint8 and workspace.dim() == 1 and workspace.is_contiguous()
              and workspace.numel() >= need and workspace.get_device() == dev)
        for i, n in enumerate(cols):
            s, d = y[i], out[i]
            ok = (ok and s.dtype is _BF16 and s.shape == (rows, n) and s.is_contiguous() and s.get_device() == dev
                  and (d is s or (d.dtype is _BF16 and d.shape == (rows, n) and d.is_contiguous()
                                  and d.get_device() == dev)))
            src.append(s.data_ptr())
            dst.append(d.data_ptr())
    except (AttributeError, TypeError, IndexError):
        ok = False
    if not ok:
        for name, ts in (("y", y), ("out", out)):
            if not isinstance(ts, (list, tuple)) or len(ts) != len(cols):
                raise ValueError(f"{name} must be a list of {len(cols)} tensors")
        if isinstance(workspace, torch.Tensor) and workspace.numel() < need:
            raise ValueError(f"workspace has {workspace.numel()} bytes, the plan needs {need}")
        _refuse(("x", x, _BF16, (rows, pool.K)),
                *((f"{name}[{i}]", t, _BF16, (rows, n)) for name, ts in (("y", y), ("out", out))
                  for i, (t, n) in enumerate(zip(ts, cols))),
                ("workspace", workspace, torch.uint8, (_numel(workspace),)), ("the pool", pool.tensors[0], _BF16,
                                                                             pool.tensors[0].shape))
    if rows == 0:
        return
    try:
        at = ctypes.byref(_CHAR.from_buffer(plan))
    except TypeError:                                # (read-only)
        at = plan.ctypes.data
    none = (0,) * (3 - len(cols))
    st = (_lib or load()).hb_adapters(ctypes.byref(pool), at, x.data_ptr(), _LINEAR_OUT.pack(*src, *none, *cols, *none),
                                      _LINEAR_OUT.pack(*dst, *none, *cols, *none), workspace.data_ptr(),
                                      _raw_stream(stream, dev))
    if st:
        _check(st)
