"""Python binding of libdfv.so.  Argument marshalling only: every step of the
block-verify path runs in the library's CUDA kernels.  Tensors must be CUDA
tensors; calls enqueue work on torch's current CUDA stream, or on the one given
as `stream` (a result that the call makes is then in that stream's memory, as
under torch.cuda.stream(stream)).  The block-verify
calls go through ctypes; the tree-verify and prompt calls, which a step makes dozens of,
through the extension built from csrc/binding.cpp."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
from typing import Optional, Sequence

import torch

from .inputs import LayerWeights

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdfv.so")
BIND_PATH = os.path.join(HERE, "_dfvbind.so")

F32, BF16, MXFP4, Q8, F16, E4M3 = 0, 1, 2, 3, 4, 5
# device error bits (DFV_DEVERR_* in include/dfv.h)
DEVERR_STAGE_WAIT, DEVERR_SLOT_WAIT, DEVERR_DRAIN_WAIT, DEVERR_GRID_WAIT = 0x1, 0x2, 0x4, 0x8
DEVERR_SCALE_RANGE, DEVERR_REDUCE_WAIT, DEVERR_ROUTING = 0x10, 0x20, 0x40
# cache error bits (DFV_KVERR_* in include/dfv.h)
KVERR_PAGE, KVERR_LEN, KVERR_NO_PAGE, KVERR_PATH, KVERR_SEQ = 0x1, 0x2, 0x4, 0x8, 0x10
MAX_TREE, MAX_TREE_SEQS, MAX_ROWS = 64, 1024, 1 << 24
_NAMES = {"f32": F32, "bf16": BF16, "mxfp4": MXFP4, "q8": Q8}
EXPORTS = ("dfv_version", "dfv_status_string", "dfv_last_error_detail", "dfv_profile_set_events",
           "dfv_read_device_error", "dfv_set_path", "dfv_last_layer_path", "dfv_fused_unavailable_reason",
           "dfv_accept_greedy_noalloc", "dfv_set_staging", "dfv_last_staging",
           "dfv_moe_workspace_size",
           "dfv_route_topk", "dfv_moe_block_forward", "dfv_moe_block_forward_host", "dfv_moe_stack_forward",
           "dfv_accept_workspace_size", "dfv_accept_greedy", "dfv_selftest_bounded_waits", "dfv_selftest_mma",
           "dfv_selftest_tcgen05", "dfv_moe_batch_workspace_size", "dfv_moe_batch_forward",
           "dfv_set_stack_launch",
           "dfv_rope_table", "dfv_rope_append", "dfv_tree_attention_workspace_size", "dfv_tree_attention",
           "dfv_logits_workspace_size", "dfv_logits_process", "dfv_accept_tree", "dfv_cache_workspace_size",
           "dfv_cache_commit", "dfv_cache_copy_pages", "dfv_pages_reserve", "dfv_pages_fork", "dfv_pages_free",
           "dfv_norm_rope_append", "dfv_cache_read", "dfv_prompt_attention_workspace_size", "dfv_prompt_attention")


class DfvError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _load()
        super().__init__("%s: %s: %s" % (where, lib.dfv_status_string(status).decode(),
                                         lib.dfv_last_error_detail().decode()))
        self.status = status


class CLayer(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int), ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int),
        ("d_ff", ctypes.c_int), ("norm_topk", ctypes.c_int),
        ("w_dtype", ctypes.c_int), ("r_dtype", ctypes.c_int),
        ("w_router", ctypes.c_void_p), ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
        ("w_down", ctypes.c_void_p), ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p),
        ("s_down", ctypes.c_void_p), ("n_shared", ctypes.c_int),
    ]


class CCache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("n_layers", "n_pages", "page_size", "n_kv_heads", "head_dim", "dtype",
                                             "max_seqs", "max_pages")]
                + [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]
                + [(n, ctypes.c_int64) for n in ("stride_layer", "stride_page", "stride_head", "stride_token")]
                + [(n, ctypes.c_void_p) for n in ("page_table", "lens", "refs", "err", "k_exp", "v_exp")])


class CTree(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("n_rows", ctypes.c_int), ("max_nodes", ctypes.c_int),
                ("seq", ctypes.c_void_p), ("row_off", ctypes.c_void_p), ("mask", ctypes.c_void_p)]


class CRows(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("n_rows", ctypes.c_int), ("max_rows", ctypes.c_int),
                ("seq", ctypes.c_void_p), ("row_off", ctypes.c_void_p)]


class CRules(ctypes.Structure):
    _fields_ = [("hist", ctypes.c_void_p), ("hist_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p),
                ("hist_row", ctypes.c_int64), ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("bias_row", ctypes.c_int64),
                ("allowed", ctypes.c_void_p), ("allowed_row", ctypes.c_int64)]


# the descriptors with what the extension's checks need beside them (csrc/binding.cpp)
class CCacheHandle(ctypes.Structure):
    _fields_ = [("c", CCache), ("index", ctypes.c_int)]


class CTreeHandle(ctypes.Structure):
    _fields_ = [("c", CTree), ("index", ctypes.c_int)]


class CRowsHandle(ctypes.Structure):
    _fields_ = [("c", CRows), ("index", ctypes.c_int)]


class CRulesHandle(ctypes.Structure):
    _fields_ = [("c", CRules), ("n_seqs", ctypes.c_int), ("index", ctypes.c_int), ("bias_rows", ctypes.c_int),
                ("allowed_rows", ctypes.c_int), ("bias_cols", ctypes.c_int64), ("allowed_cols", ctypes.c_int64)]


_lib = None


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libdfv.so is not built (%s); run speculative_decoding_moe_gb300.build.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.dfv_version.restype = I
        L.dfv_status_string.restype = ctypes.c_char_p
        L.dfv_status_string.argtypes = [I]
        L.dfv_last_error_detail.restype = ctypes.c_char_p
        L.dfv_moe_workspace_size.restype = S
        L.dfv_moe_workspace_size.argtypes = [P, I]
        L.dfv_route_topk.argtypes = [P, P, I, I, P, P, P, P, P, P, P, S, P]
        L.dfv_moe_block_forward.argtypes = [P, P, I, I, P, P, P, P, S, P]
        L.dfv_moe_block_forward_host.argtypes = [P, P, I, I, P, P, S, P]
        L.dfv_moe_stack_forward.argtypes = [P, I, P, I, ctypes.c_float, P, P, S, P]
        L.dfv_accept_workspace_size.restype = S
        L.dfv_accept_workspace_size.argtypes = [I, I]
        L.dfv_accept_greedy.argtypes = [P, I, I, I, P, P, P, P, S, P]
        L.dfv_profile_set_events.argtypes = [P, I]
        L.dfv_accept_greedy_noalloc.argtypes = [P, I, I, I, P, P, P, P]
        L.dfv_read_device_error.argtypes = [P, P, P]
        L.dfv_selftest_bounded_waits.argtypes = [P, S, P]
        L.dfv_selftest_mma.argtypes = [I, P, P, P, P]
        L.dfv_selftest_tcgen05.argtypes = [P, P, I, I, P, P, P]
        L.dfv_moe_batch_workspace_size.restype = S
        L.dfv_moe_batch_workspace_size.argtypes = [P, I]
        L.dfv_moe_batch_forward.argtypes = [P, P, I, I, P, P, P, P, S, P]
        L.dfv_set_path.argtypes = [I]
        L.dfv_set_stack_launch.argtypes = [I]
        L.dfv_set_staging.restype = I
        L.dfv_set_staging.argtypes = [I]
        L.dfv_last_staging.restype = I
        L.dfv_last_staging.argtypes = []
        L.dfv_last_layer_path.restype = I
        L.dfv_fused_unavailable_reason.restype = ctypes.c_char_p
        F, F64, L64 = ctypes.c_float, ctypes.c_double, ctypes.c_int64
        L.dfv_rope_table.argtypes = [I, F64, I, F64, F64, F64, F64, P]
        L.dfv_rope_append.argtypes = [P, I, P, I, I, I, F, P, P, L64, L64, P, L64, L64, P, L64, L64, P, P, L64, L64, P]
        L.dfv_tree_attention_workspace_size.restype = S
        L.dfv_tree_attention_workspace_size.argtypes = [P, P, I]
        L.dfv_tree_attention.argtypes = [P, I, P, I, F, P, L64, L64, P, L64, L64, P, P, S, P]
        L.dfv_logits_workspace_size.restype = S
        L.dfv_logits_workspace_size.argtypes = [I]
        L.dfv_logits_process.argtypes = [P, L64, I, I, P, P, P, P, L64, P, P, S, P]
        L.dfv_accept_tree.argtypes = [P, P, P, P, L64, P, P]
        L.dfv_cache_workspace_size.restype = S
        L.dfv_cache_workspace_size.argtypes = [P]
        L.dfv_cache_commit.argtypes = [P, P, P, L64, P, P, P, S, P]
        L.dfv_cache_copy_pages.argtypes = [P, P, P, I, P]
        L.dfv_pages_reserve.argtypes = [P, P, P, I, P, S, P]
        L.dfv_pages_fork.argtypes = [P, P, P, I, P, S, P]
        L.dfv_pages_free.argtypes = [P, P, I, P]
        L.dfv_norm_rope_append.argtypes = [P, I, P, I, P, P, F, I, I, F, P, P, L64, L64, P, L64, L64, P, L64, L64, P, P, L64, L64, P, L64, L64, P]
        L.dfv_cache_read.argtypes = [P, I, P, P, L64, L64, P, L64, L64, P]
        L.dfv_prompt_attention_workspace_size.restype = S
        L.dfv_prompt_attention_workspace_size.argtypes = [P, I, I, I]
        L.dfv_prompt_attention.argtypes = [I, P, P, I, I, I, F, P, L64, L64, P, L64, L64, P, L64, L64, P, L64, L64, P, P, P, S, P]
        _lib = L
    return _lib


_ext = None


def _bind():
    """The extension with the tree-verify and prompt calls."""
    global _ext
    if _ext is None:
        _load()
        if not os.path.exists(BIND_PATH):
            raise ImportError("_dfvbind.so is not built (%s); run speculative_decoding_moe_gb300.build.build()" % BIND_PATH)
        loader = importlib.machinery.ExtensionFileLoader("_dfvbind", BIND_PATH)
        spec = importlib.util.spec_from_file_location("_dfvbind", BIND_PATH, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _ext = module
    return _ext


def lib():
    return _load()


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A result, in the memory of the call's stream: a block of the current stream's may still be in use there, and would
    be handed out there again before the call ends."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _act(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("activations must be bf16 or fp32, got %s" % t.dtype)


def _check(status: int, where: str):
    if status != 0:
        raise DfvError(status, where)


class Layer:
    """A layer descriptor over device-resident weights (keeps them alive)."""

    def __init__(self, w: LayerWeights):
        for t in (w.w_router, w.w_gate, w.w_up, w.w_down):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("layer weights must be contiguous CUDA tensors")
        s = w.shape
        if w.w_gate.shape[0] != s.n_experts + s.n_shared:
            raise ValueError("expert matrices hold %d experts, the shape needs %d routed + %d shared"
                             % (w.w_gate.shape[0], s.n_experts, s.n_shared))
        self.w = w
        self.shape = s
        self.c = CLayer(s.d, s.n_experts, s.top_k, s.d_ff, s.norm_topk, _NAMES[s.w_dtype], _NAMES[s.r_dtype],
                        w.w_router.data_ptr(), w.w_gate.data_ptr(), w.w_up.data_ptr(), w.w_down.data_ptr(),
                        None if w.s_gate is None else w.s_gate.data_ptr(),
                        None if w.s_up is None else w.s_up.data_ptr(),
                        None if w.s_down is None else w.s_down.data_ptr(), s.n_shared)

    @property
    def ref(self):
        return ctypes.byref(self.c)


def workspace_size(layer: Layer, k_max: int) -> int:
    return int(_load().dfv_moe_workspace_size(layer.ref, int(k_max)))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Zero-filled workspace (the library requires zeros before first use).  One may serve several calls in stream order
    if they are of one family: the MoE block and stack calls, the batched ones, accept_greedy, or all tree-verify and prompt calls."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def route_topk(layer: Layer, hidden: torch.Tensor, ws: torch.Tensor, stream=None):
    k = hidden.shape[0]
    s = layer.shape
    dev = hidden.device
    ints = lambda *shape: _empty(shape, torch.int32, dev, stream)  # noqa: E731
    idx = ints(k, s.top_k)
    w = _empty((k, s.top_k), torch.float32, dev, stream)
    woken = ints(min(s.n_experts, k * s.top_k))
    nw = ints(1)
    offs = ints(min(s.n_experts, k * s.top_k) + 1)
    gat = ints(k * s.top_k)
    st = _load().dfv_route_topk(layer.ref, _p(hidden), _act(hidden), k, _p(idx), _p(w), _p(woken), _p(nw), _p(offs),
                                _p(gat), _p(ws), ws.numel(), _stream(stream))
    _check(st, "dfv_route_topk")
    return dict(topk_idx=idx, topk_w=w, woken=woken, n_woken=nw, offsets=offs, gather=gat)


def moe_block_forward(layer: Layer, hidden: torch.Tensor, ws: torch.Tensor, out: Optional[torch.Tensor] = None,
                      topk_idx: Optional[torch.Tensor] = None, n_woken: Optional[torch.Tensor] = None, stream=None):
    k = hidden.shape[0]
    if out is None:
        out = torch.empty_like(hidden) if stream is None else _empty(hidden.shape, hidden.dtype, hidden.device, stream)
    st = _load().dfv_moe_block_forward(layer.ref, _p(hidden), _act(hidden), k, _p(out), _p(topk_idx), _p(n_woken),
                                       _p(ws), ws.numel(), _stream(stream))
    _check(st, "dfv_moe_block_forward")
    return out


def batch_workspace_size(layer: Layer, n_rows_max: int) -> int:
    return int(_load().dfv_moe_batch_workspace_size(layer.ref, int(n_rows_max)))


def moe_batch_forward(layer: Layer, hidden: torch.Tensor, n_blocks: int, ws: torch.Tensor,
                      out: Optional[torch.Tensor] = None, topk_idx: Optional[torch.Tensor] = None,
                      n_woken: Optional[torch.Tensor] = None, stream=None):
    """n_blocks verify blocks of k = rows / n_blocks positions through one layer."""
    T = hidden.shape[0]
    if T % n_blocks:
        raise ValueError("rows %d are not n_blocks=%d blocks of equal size" % (T, n_blocks))
    if out is None:
        out = torch.empty_like(hidden) if stream is None else _empty(hidden.shape, hidden.dtype, hidden.device, stream)
    st = _load().dfv_moe_batch_forward(layer.ref, _p(hidden), n_blocks, T // n_blocks, _p(out), _p(topk_idx),
                                       _p(n_woken), _p(ws), ws.numel(), _stream(stream))
    _check(st, "dfv_moe_batch_forward")
    return out


def moe_block_forward_host(layer: Layer, hidden_host: torch.Tensor, out_host: torch.Tensor, ws: torch.Tensor,
                           stream=None):
    """hidden_host / out_host: CPU tensors (pinned for asynchronous copies)."""
    k = hidden_host.shape[0]
    st = _load().dfv_moe_block_forward_host(layer.ref, _p(hidden_host), _act(hidden_host), k, _p(out_host), _p(ws),
                                            ws.numel(), _stream(stream))
    _check(st, "dfv_moe_block_forward_host")
    return out_host


def moe_stack_forward(layers: Sequence[Layer], x: torch.Tensor, ws: torch.Tensor, eps: float = 1e-6, stream=None,
                      n_woken: Optional[torch.Tensor] = None):
    """x <- the stack applied to x (in place).  n_woken: optional int32 [len(layers)]
    device tensor that receives each layer's routed woken-expert count."""
    arr = (CLayer * len(layers))(*[L.c for L in layers])
    if n_woken is not None and (n_woken.dtype != torch.int32 or n_woken.numel() < len(layers)):
        raise ValueError("n_woken must be int32 with one entry per layer")
    st = _load().dfv_moe_stack_forward(arr, len(layers), _p(x), x.shape[0], float(eps), _p(n_woken), _p(ws),
                                       ws.numel(), _stream(stream))
    _check(st, "dfv_moe_stack_forward")
    return x


def accept_workspace_size(k_max: int, V: int) -> int:
    return int(_load().dfv_accept_workspace_size(int(k_max), int(V)))


def accept_greedy(logits: torch.Tensor, draft: torch.Tensor, ws: torch.Tensor, tau: Optional[torch.Tensor] = None,
                  committed: Optional[torch.Tensor] = None, stream=None):
    rows, V = logits.shape
    k = rows - 1
    dev = logits.device
    if tau is None:
        tau = _empty(1, torch.int32, dev, stream)
    if committed is None:
        committed = _empty(k + 1, torch.int32, dev, stream)
    st = _load().dfv_accept_greedy(_p(logits), _act(logits), k, V, _p(draft), _p(tau), _p(committed), _p(ws),
                                   ws.numel(), _stream(stream))
    _check(st, "dfv_accept_greedy")
    return tau, committed


def profile_set_events(events: Optional[Sequence[torch.cuda.Event]]):
    """Record the 4 phase-boundary events in later layer calls (None: off)."""
    if events is None:
        _check(_load().dfv_profile_set_events(None, 0), "dfv_profile_set_events")
        return
    for e in events:
        if e.cuda_event == 0:  # torch creates the CUDA event on first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(_load().dfv_profile_set_events(arr, len(events)), "dfv_profile_set_events")


def read_device_error(ws: torch.Tensor, stream=None) -> int:
    """Device error bits of a workspace (synchronises the stream)."""
    out = ctypes.c_uint32(0)
    _check(_load().dfv_read_device_error(_p(ws), ctypes.byref(out), _stream(stream)), "dfv_read_device_error")
    (stream if stream is not None else torch.cuda.current_stream()).synchronize()
    return int(out.value)


def selftest_bounded_waits(ws: torch.Tensor, stream=None):
    """Run the bounded-wait self-test on `ws` (about 4 s on the GPU; read the
    error word with read_device_error, then zero-fill ws)."""
    _check(_load().dfv_selftest_bounded_waits(_p(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "dfv_selftest_bounded_waits")


def selftest_mma(a: torch.Tensor, b: torch.Tensor, stream=None) -> torch.Tensor:
    """D = A . B (16 x 16 x 16) through the expert kernels' MMA fragment path;
    a and b are bf16 or fp16 CUDA tensors [16, 16]."""
    if a.shape != (16, 16) or b.shape != (16, 16) or a.dtype != b.dtype:
        raise ValueError("A and B must be [16, 16] tensors of one dtype")
    code = {torch.bfloat16: BF16, torch.float16: F16}.get(a.dtype)
    if code is None:
        raise TypeError("A and B must be bf16 or fp16, got %s" % a.dtype)
    a, b = a.contiguous(), b.contiguous()
    out = torch.empty(16, 16, dtype=torch.float32, device=a.device)
    _check(_load().dfv_selftest_mma(code, _p(a), _p(b), _p(out), _stream(stream)), "dfv_selftest_mma")
    return out


def selftest_tcgen05(a: torch.Tensor, b: torch.Tensor, stream=None):
    """D = A . B^T (A [128, K], B [N, K], bf16) through the tcgen05 / TMEM path;
    returns (D [128, N] fp32, status)."""
    if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16 or a.shape[0] != 128 or a.shape[1] != b.shape[1]:
        raise ValueError("A must be [128, K] and B [N, K], both bf16")
    a, b = a.contiguous(), b.contiguous()
    d = torch.full((128, b.shape[0]), float("nan"), dtype=torch.float32, device=a.device)
    st = torch.zeros(1, dtype=torch.int32, device=a.device)
    _check(_load().dfv_selftest_tcgen05(_p(a), _p(b), b.shape[0], a.shape[1], _p(d), _p(st), _stream(stream)),
           "dfv_selftest_tcgen05")
    return d, st


def set_staging(max_mode: int):
    """Highest gate/up staging mode of the single-launch bf16 kernel (3, the default, 2, 1 or 0)."""
    _check(_load().dfv_set_staging(int(max_mode)), "dfv_set_staging")


def last_staging() -> int:
    return int(_load().dfv_last_staging())


def set_path(fused: bool):
    """Select the fused single-launch layer kernel (default) or the multi-kernel path."""
    _check(_load().dfv_set_path(1 if fused else 0), "dfv_set_path")


def set_stack_launch(mode):
    """Stacks whose layers allow it: 0 (or False) one launch per layer; 1 (default) one persistent
    launch per 48 layers for eager calls with k <= 8 (per layer inside a CUDA graph); 2 (or True)
    one persistent launch per 48 layers for every k."""
    m = {False: 0, True: 2}.get(mode, mode) if isinstance(mode, bool) else int(mode)
    _check(_load().dfv_set_stack_launch(m), "dfv_set_stack_launch")


def last_layer_path() -> int:
    """Path of the last layer call from this thread: 1 fused, 0 multi-kernel, 2 batched, 3 persistent stack."""
    return int(_load().dfv_last_layer_path())


def fused_unavailable_reason() -> str:
    return _load().dfv_fused_unavailable_reason().decode()


def accept_greedy_noalloc(logits: torch.Tensor, draft: torch.Tensor, tau: Optional[torch.Tensor] = None,
                          committed: Optional[torch.Tensor] = None, stream=None):
    """Greedy acceptance with the library's fixed device scratch (no workspace)."""
    rows, V = logits.shape
    k = rows - 1
    dev = logits.device
    if tau is None:
        tau = _empty(1, torch.int32, dev, stream)
    if committed is None:
        committed = _empty(k + 1, torch.int32, dev, stream)
    st = _load().dfv_accept_greedy_noalloc(_p(logits), _act(logits), k, V, _p(draft), _p(tau), _p(committed),
                                           _stream(stream))
    _check(st, "dfv_accept_greedy_noalloc")
    return tau, committed


# ---------------------------------------------------------------- tree verify
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _on(stream, index: int) -> int:
    """Stream handle of a call: the given stream, or torch's current one.  The library launches on the current device."""
    if index < 0:
        return 0  # host tensors are refused by the call
    if index != _current_device():
        raise ValueError("the tensors of the call are on device %d, the current device is %d" % (index, _current_device()))
    if stream is None:
        return _raw_stream(index)
    if stream.device_index != index:
        raise ValueError("the tensors of the call are on device %d, the stream is on device %d" % (index, stream.device_index))
    return stream.cuda_stream


def _refuse(t, what: str, dtype, shape, index: int):
    if t is None:
        raise ValueError("%s is missing" % what)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s is on %s, not with the other tensors of the call" % (what, t.device))
    raise ValueError("%s must be contiguous" % what)


def _need(t: Optional[torch.Tensor], what: str, dtype, shape, index: int) -> int:
    """Address of a contiguous tensor of this type and shape on this device."""
    if t is None or t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        _refuse(t, what, dtype, shape, index)
    return t.data_ptr()


def _given(t: Optional[torch.Tensor], what: str, dtype, shape, index: int) -> Optional[int]:
    """_need for an argument that may be left out."""
    return None if t is None else _need(t, what, dtype, shape, index)


class KVCache:
    """A paged key/value cache of all layers (include/dfv.h, dfv_kv_cache).

    k, v        [n_layers, n_pages, n_kv_heads, page_size, head_dim] bf16, fp16 or float8_e4m3fn, any strides that both
                share with the last dimension contiguous (permuted views of token-major pages, halves of one allocation)
    page_table  [max_seqs, max_pages] int32, -1 where there is no page
    lens        [max_seqs] int32 committed tokens
    refs        [n_pages] int32 holders of each page, 0 = free (for the page calls)
    err         [1] int32 error bits (KVERR_*), sticky; made here when not given
    k_exp, v_exp [n_layers, n_pages, n_kv_heads, page_size] uint8, for float8_e4m3fn: a token's values are its codes
                times 2^(exp - 127); rows in and out of such a cache are bf16
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                 refs: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                 k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None):
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be alike: [layers, pages, kv heads, page size, head dim]")
        kind = {torch.bfloat16: BF16, torch.float16: F16, torch.float8_e4m3fn: E4M3}.get(k.dtype)
        if kind is None:
            raise TypeError("the cache must be bf16, fp16 or float8_e4m3fn, got %s" % k.dtype)
        if k.stride(4) != 1 or v.stride(4) != 1 or any(a != b for a, b, n in zip(k.stride(), v.stride(), k.shape) if n > 1):
            raise ValueError("k and v must have the same strides and a contiguous head dimension")
        at = k.get_device()
        if kind == E4M3:
            _need(k_exp, "k_exp", torch.uint8, k.shape[:4], at)
            _need(v_exp, "v_exp", torch.uint8, k.shape[:4], at)
        elif k_exp is not None or v_exp is not None:
            raise ValueError("k_exp and v_exp belong to a float8_e4m3fn cache, this one is %s" % k.dtype)
        if page_table.dim() != 2:
            raise ValueError("page_table must be [max_seqs, max_pages], got %s" % (tuple(page_table.shape),))
        _need(page_table, "page_table", torch.int32, page_table.shape, at)
        _need(lens, "lens", torch.int32, page_table.shape[:1], at)
        _given(refs, "refs", torch.int32, k.shape[1:2], at)
        if err is None:
            err = torch.zeros(1, dtype=torch.int32, device=k.device)
        _need(err, "err", torch.int32, (1,), at)
        self.index = at
        self.k, self.v, self.page_table, self.lens, self.refs, self.err = k, v, page_table, lens, refs, err
        self.k_exp, self.v_exp = k_exp, v_exp
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.dtype = k.dtype
        st = [k.stride(i) if k.shape[i] > 1 else 0 for i in range(4)]
        self.c = CCache(self.n_layers, self.n_pages, self.page_size, self.n_kv_heads, self.head_dim,
                        kind, page_table.shape[0], page_table.shape[1],
                        k.data_ptr(), v.data_ptr(), st[0], st[1], st[2], k.stride(3) if self.page_size > 1 else self.head_dim,
                        page_table.data_ptr(), lens.data_ptr(), None if refs is None else refs.data_ptr(),
                        err.data_ptr(), None if k_exp is None else k_exp.data_ptr(), None if v_exp is None else v_exp.data_ptr())
        self._handle = CCacheHandle(self.c, at)
        self.c = self._handle.c
        self.ref = ctypes.byref(self.c)
        self.addr = ctypes.addressof(self._handle)

    @classmethod
    def empty(cls, n_layers: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, max_seqs: int,
              max_pages: int, dtype=torch.bfloat16, device="cuda") -> "KVCache":
        """An empty cache: every page free, every sequence without tokens."""
        kv = torch.zeros(2, n_layers, n_pages, n_kv_heads, page_size, head_dim, dtype=dtype, device=device)
        exp = [None, None]
        if dtype == torch.float8_e4m3fn:
            exp = torch.full((2, n_layers, n_pages, n_kv_heads, page_size), 127, dtype=torch.uint8, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        return cls(kv[0], kv[1], torch.full((max_seqs, max_pages), -1, **i32), torch.zeros(max_seqs, **i32),
                   refs=torch.zeros(n_pages, **i32), k_exp=exp[0], v_exp=exp[1])

    def errors(self) -> int:
        """Error bits so far (waits for the device)."""
        return int(self.err.item()) & 0xffffffff


class TreeBatch:
    """The drafted trees of one call (include/dfv.h, dfv_tree_batch): n_rows nodes, sequence b's in rows
    row_off[b] .. row_off[b + 1], at most max_nodes each; mask [n_rows] int64 bit patterns (None: chains); seq
    [n_seqs] int32 cache sequences (None: 0, 1, ...)."""

    def __init__(self, row_off: torch.Tensor, n_rows: int, max_nodes: int, mask: Optional[torch.Tensor] = None,
                 seq: Optional[torch.Tensor] = None):
        if row_off.dim() != 1 or row_off.numel() < 2:
            raise ValueError("row_off needs one entry per sequence and one more")
        at = row_off.get_device()
        _need(row_off, "row_off", torch.int32, row_off.shape, at)
        self.n_seqs, self.n_rows, self.max_nodes = row_off.numel() - 1, int(n_rows), int(max_nodes)
        _given(mask, "mask", torch.int64, (self.n_rows,), at)
        _given(seq, "seq", torch.int32, (self.n_seqs,), at)
        self.index = at
        self.row_off, self.mask, self.seq = row_off, mask, seq
        self.c = CTree(self.n_seqs, self.n_rows, self.max_nodes, None if seq is None else seq.data_ptr(),
                       row_off.data_ptr(), None if mask is None else mask.data_ptr())
        self._handle = CTreeHandle(self.c, at)
        self.c = self._handle.c
        self.ref = ctypes.byref(self.c)
        self.addr = ctypes.addressof(self._handle)


class RowBatch:
    """The rows of one call, any number per sequence (include/dfv.h, dfv_row_batch): sequence b's are rows row_off[b] ..
    row_off[b + 1] of n_rows, at most max_rows; seq [n_seqs] int32 cache sequences (None: 0, 1, ...)."""

    def __init__(self, row_off: torch.Tensor, n_rows: int, max_rows: int, seq: Optional[torch.Tensor] = None):
        if row_off.dim() != 1 or row_off.numel() < 2:
            raise ValueError("row_off needs one entry per sequence and one more")
        at = row_off.get_device()
        _need(row_off, "row_off", torch.int32, row_off.shape, at)
        self.n_seqs, self.n_rows, self.max_rows = row_off.numel() - 1, int(n_rows), int(max_rows)
        _given(seq, "seq", torch.int32, (self.n_seqs,), at)
        self.index = at
        self.row_off, self.seq = row_off, seq
        self.c = CRows(self.n_seqs, self.n_rows, self.max_rows, None if seq is None else seq.data_ptr(), row_off.data_ptr())
        self._handle = CRowsHandle(self.c, at)
        self.c = self._handle.c
        self.ref = ctypes.byref(self.c)
        self.rows_addr = ctypes.addressof(self._handle)  # (not `addr`: a TreeBatch is another descriptor)


class Rope:
    """Rotary plan: the device table of dfv_rope_table and the factor on cos and sin.

    scaling: "none", "linear", "ntk" or "bands" (frequency bands between `low` and `high` turns over the `original`
    context; attention is then scaled by 0.1 ln(factor) + 1 unless `scale` says otherwise).  "bands" ramps linearly in the
    turns; a model whose configuration means another ramp (linear in the pair's index between two rounded indexes, say)
    has other frequencies in between, by tens of percent: those go in as
    freqs: the rot_dim / 2 angles per position of the pairs, in place of theta and scaling (scale: 1 unless given)."""

    KINDS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3}

    def __init__(self, head_dim: int, rot_dim: Optional[int] = None, theta: float = 1e4, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original: int = 4096, low: float = 1.0, high: float = 32.0,
                 scale: Optional[float] = None, device="cuda", freqs: Optional[Sequence[float]] = None):
        if scaling not in self.KINDS:
            raise ValueError("scaling must be one of %s, got %r" % (sorted(self.KINDS), scaling))
        self.head_dim, self.interleaved = int(head_dim), int(bool(interleaved))
        self.rot_dim = self.head_dim if rot_dim is None else int(rot_dim)
        turns = (ctypes.c_uint64 * max(1, self.rot_dim // 2))()
        _check(_load().dfv_rope_table(self.rot_dim, float(theta), self.KINDS[scaling], float(factor), float(original),
                                      float(low), float(high), turns), "dfv_rope_table")
        if freqs is not None:
            freqs = [float(f) for f in freqs]
            if len(freqs) != self.rot_dim // 2 or not all(map(math.isfinite, freqs)):
                raise ValueError("freqs must be rot_dim / 2 = %d finite angles, got %d" % (self.rot_dim // 2, len(freqs)))
            if scaling != "none":
                raise ValueError("freqs are taken as they are: scaling must be 'none'")
            turns = [round(math.ldexp(f / (2 * math.pi), 64)) % (1 << 64) for f in freqs]
        if scale is None:
            scale = 0.1 * math.log(factor) + 1.0 if scaling == "bands" else 1.0
        self.scale = float(scale)
        signed = [t - (1 << 64) if t >> 63 else t for t in turns]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)
        self.turns_addr, self.index = self.turns.data_ptr(), self.turns.get_device()


def rope_append(cache: KVCache, layer: int, tree: TreeBatch, rope: Rope, q: torch.Tensor, k: torch.Tensor,
                v: torch.Tensor, positions: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotated q (out, a new tensor or q itself), and the rows' rotated k and their v stored into the cache.
    q [rows, heads, dim], k and v [rows, kv heads, dim] may be slices of one projection."""
    return (_ext or _bind()).rope_append(cache.addr, layer, tree.addr, rope.head_dim, rope.rot_dim, rope.interleaved,
                                         rope.scale, rope.turns_addr, q, k, v, positions, out,
                                         _on(stream, cache.index), rope.index)


def norm_rope_append(cache: KVCache, layer: int, rows: RowBatch, rope: Rope, q: torch.Tensor, k: torch.Tensor,
                     v: torch.Tensor, positions: torch.Tensor, q_gain: Optional[torch.Tensor] = None,
                     k_gain: Optional[torch.Tensor] = None, eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                     k_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Normed and rotated q (out, a new tensor or q itself), and the rows' normed and rotated k and their v stored into
    the cache behind the committed tokens, for any number of rows.  q_gain, k_gain [dim]: the gains of the norm over each
    head's elements (None: no norm); q [rows, heads, dim], k and v [rows, kv heads, dim] may be slices of one projection.
    k_out: optional rows that receive the normed and rotated k too (k itself is fine), for prompt_attention."""
    return (_ext or _bind()).norm_rope_append(cache.addr, layer, rows.rows_addr, rope.head_dim, rope.rot_dim, rope.interleaved,
                                              rope.scale, rope.turns_addr, q, k, v, positions, q_gain, k_gain, eps, out,
                                              _on(stream, cache.index), rope.index, k_out)


def cache_read(cache: KVCache, layer: int, rows: RowBatch, k: Optional[torch.Tensor] = None,
               v: Optional[torch.Tensor] = None, stream=None):
    """(k, v) [rows, kv heads, dim]: row i of a sequence is its token i in the cache, counted from its first one (tokens
    that were appended but not committed yet too); a float8_e4m3fn cache gives bf16."""
    return (_ext or _bind()).cache_read(cache.addr, layer, rows.rows_addr, cache.k, k, v, _on(stream, cache.index))


def prompt_attention_workspace_size(rows: RowBatch, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(_load().dfv_prompt_attention_workspace_size(rows.ref, int(n_heads), int(n_kv_heads), int(head_dim)))


def prompt_attention(rows: RowBatch, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, ws: torch.Tensor,
                     keys: Optional[RowBatch] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of packed prompts: q [rows, heads, dim] over k, v [key rows, kv heads, dim], bf16 or fp16.
    keys: the key rows of each sequence when they are not its q rows (the q rows are then the last of them); scale:
    1/sqrt(dim) by default; lse: optional fp32 [rows, heads] that receives ln(sum exp); err: optional int32 [1] that
    receives KVERR_LEN for offsets out of range."""
    return (_ext or _bind()).prompt_attention(rows.rows_addr, 0 if keys is None else keys.rows_addr, q, k, v, ws, scale, out, lse, err,
                                              _on(stream, rows.index))


def tree_attention_workspace_size(cache: KVCache, tree: TreeBatch, n_heads: int) -> int:
    return int(_load().dfv_tree_attention_workspace_size(cache.ref, tree.ref, int(n_heads)))


def tree_attention(cache: KVCache, layer: int, tree: TreeBatch, q: torch.Tensor, ws: torch.Tensor,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of every drafted node over its sequence's committed tokens and the nodes of its mask.
    scale: 1/sqrt(head_dim) by default; lse: optional fp32 [rows, heads] that receives ln(sum exp)."""
    return (_ext or _bind()).tree_attention(cache.addr, layer, tree.addr, q, ws, scale, out, lse, _on(stream, cache.index))


class LogitRules:
    """Penalties, bias and grammar mask of a call (include/dfv.h, dfv_logit_rules); any of them may be None.

    hist [n_seqs, width] int32 with hist_len, prompt_len [n_seqs] int32; repetition, frequency, presence [n_seqs]
    fp32; bias [n_seqs or 1, V] fp32; allowed [rows or 1, ceil(V / 32)] int32 bit words."""

    def __init__(self, hist=None, hist_len=None, prompt_len=None, repetition=None, frequency=None, presence=None,
                 bias=None, allowed=None):
        given = [t for t in (hist, hist_len, prompt_len, repetition, frequency, presence, bias, allowed) if t is not None]
        at = given[0].get_device() if given else None
        for name, t, dt in (("hist", hist, torch.int32), ("bias", bias, torch.float32), ("allowed", allowed, torch.int32)):
            if t is not None and t.dim() != 2:
                raise ValueError("%s must have two dimensions, got %s" % (name, tuple(t.shape)))
            _given(t, name, dt, None if t is None else t.shape, at)
        if hist is not None and hist_len is None:
            raise ValueError("hist needs hist_len")
        n = None if hist is None else hist.shape[0]
        for name, t, dt in (("hist_len", hist_len, torch.int32), ("prompt_len", prompt_len, torch.int32),
                            ("repetition", repetition, torch.float32), ("frequency", frequency, torch.float32),
                            ("presence", presence, torch.float32)):
            if t is not None:
                n = t.numel() if n is None else n
                _need(t, name, dt, (n,), at)
        self.index = at
        self.n_seqs, self.bias, self.allowed = n, bias, allowed
        self.keep = (hist, hist_len, prompt_len, repetition, frequency, presence)
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.c = CRules(ptr(hist), ptr(hist_len), ptr(prompt_len), 0 if hist is None else hist.shape[1], ptr(repetition),
                        ptr(frequency), ptr(presence), ptr(bias), 0 if bias is None or bias.shape[0] == 1 else bias.shape[1],
                        ptr(allowed), 0 if allowed is None or allowed.shape[0] == 1 else allowed.shape[1])
        size = lambda t: (0, 0) if t is None else tuple(t.shape)  # noqa: E731
        (br, bc), (ar, ac) = size(bias), size(allowed)
        self._handle = CRulesHandle(self.c, -1 if n is None else n, -2 if at is None else at, br, ar, bc, ac)
        self.c = self._handle.c
        self.ref = ctypes.byref(self.c)
        self.addr = ctypes.addressof(self._handle)


def logits_workspace_size(n_rows_max: int) -> int:
    return int(_load().dfv_logits_workspace_size(int(n_rows_max)))


def logits_process(logits: torch.Tensor, tree: TreeBatch, tokens: Optional[torch.Tensor], rules: LogitRules,
                   ws: torch.Tensor, out: Optional[torch.Tensor] = None, argmax: Optional[torch.Tensor] = None,
                   store: bool = True, stream=None):
    """(logits under the rules, argmax of each row).  logits [rows, V] bf16 or fp32 with contiguous rows; out may be
    logits itself; store=False computes the argmax only (out is then None)."""
    return (_ext or _bind()).logits_process(logits, tree.addr, tokens, rules.addr, ws, out, argmax, store,
                                            _on(stream, tree.index))


def accept_tree(tree: TreeBatch, tokens: torch.Tensor, target: torch.Tensor, path: Optional[torch.Tensor] = None,
                tau: Optional[torch.Tensor] = None, stream=None):
    """(path [n_seqs, max_nodes], tau [n_seqs]): the accepted nodes of each tree, root first, then -1."""
    return (_ext or _bind()).accept_tree(tree.addr, tokens, target, path, tau, _on(stream, tree.index))


def cache_workspace_size(cache: KVCache) -> int:
    return int(_load().dfv_cache_workspace_size(cache.ref))


def cache_commit(cache: KVCache, tree: TreeBatch, path: torch.Tensor, tau: torch.Tensor, ws: torch.Tensor,
                 new_lens: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the accepted rows together in every layer and adds tau to the lengths (cache.lens unless new_lens is
    given); returns the lengths."""
    return (_ext or _bind()).cache_commit(cache.addr, tree.addr, path, tau, ws, cache.lens if new_lens is None else new_lens,
                                          _on(stream, cache.index))


def cache_copy_pages(cache: KVCache, src: torch.Tensor, dst: torch.Tensor, stream=None):
    """Page dst[i] <- page src[i] in every layer."""
    (_ext or _bind()).cache_copy_pages(cache.addr, src, dst, _on(stream, cache.index))


def pages_reserve(cache: KVCache, seqs: torch.Tensor, n_new: torch.Tensor, ws: torch.Tensor, stream=None):
    """Pages for n_new[i] tokens after those of sequence seqs[i]."""
    (_ext or _bind()).pages_reserve(cache.addr, seqs, n_new, ws, _on(stream, cache.index))


def pages_fork(cache: KVCache, src: torch.Tensor, dst: torch.Tensor, ws: torch.Tensor, stream=None):
    """Sequence dst[i], which holds nothing, becomes a copy of src[i]."""
    (_ext or _bind()).pages_fork(cache.addr, src, dst, ws, _on(stream, cache.index))


def pages_free(cache: KVCache, seqs: torch.Tensor, stream=None):
    """Drops sequences: their pages lose a holder, their lengths become 0."""
    (_ext or _bind()).pages_free(cache.addr, seqs, _on(stream, cache.index))
