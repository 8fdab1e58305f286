"""tensor_transformer_layer_cube_gb300 - Python binding of ``libtp3d.so``.

The library (``include/tp3d.h``) computes the 3-D tensor-parallel linear, MLP
block and GPT decoder layer of "Maximizing Parallelism in Distributed
Training for Huge Neural Networks" over a virtual q x q x q device cube held
in one GB300's memory, plus bit-exact resharding between row, column, 2-D
block, cube and replicated layouts ("On Optimizing the Communication of Model
Parallelism", §2), in hand-written sm_103a kernels; and (``include/tp3d_plan.h``)
the host-side planners: the cross-mesh resharding planner of that page's
§3.2 and a pipeline-bubble simulator; and (``include/tp3d_paged.h``) the paged
key/value cache that serves the layer: block tables and slot maps from request
lengths, the cache write, and attention of new tokens over the cache; and
(``include/tp3d_rope.h``) the norm of query and key heads with the rotation by
position, forward and backward.

This module only marshals arguments: every function has the name of the C
entry point it calls and returns its status code (0 = TP3D_OK).  Tensor
arguments may be torch tensors (their ``data_ptr()`` is passed), raw device
pointers (int) or None.  ``stream`` may be a ``torch.cuda.Stream``, a raw
``cudaStream_t`` (int) or None for torch's current stream.  Nothing here
computes: if ``libtp3d.so`` has not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB as LIB_PATH
from .build import build

__all__ = [
    "build", "lib", "Tp3dError", "check", "STATUS", "layout",
    "tp3d_create", "tp3d_destroy", "tp3d_status_string", "tp3d_sync_status", "tp3d_reshard",
    "tp3d_set_wait_limit_ns", "tp3d_inject_load_stall",
    "tp3d_linear", "tp3d_mlp", "tp3d_mlp_plan", "tp3d_mlp_noalloc", "tp3d_layer_workspace_bytes", "tp3d_layer_fwd", "tp3d_layer_bwd",
    "tp3d_layout", "tp3d_layer_cfg", "tp3d_layer_params", "tp3d_layer_grads",
    "TP3D_F32", "TP3D_BF16", "CUBE_A", "CUBE_B", "CUBE_C", "CUBE_B_SWAP", "ROW", "COL", "BLOCK2D", "REPLICATED",
    "tp3d_rect", "tp3d_mesh_spec", "tp3d_cmr_options", "tp3d_cmr_result", "tp3d_pipe_cfg", "tp3d_pipe_op",
    "tp3d_pipe_result", "tp3d_layout_rects", "tp3d_mesh_rects", "tp3d_cmr_plan_create", "tp3d_cmr_plan_destroy",
    "tp3d_cmr_plan_num_tasks", "tp3d_cmr_plan_task", "tp3d_cmr_plan_lower_bound", "tp3d_cmr_schedule",
    "tp3d_pipeline_simulate", "tp3d_mlp_layout", "TP3D_SCHEME_1D", "TP3D_SCHEME_2D", "TP3D_SCHEME_3D", "TP3D_SPEC_R", "TP3D_SPEC_S0", "TP3D_SPEC_S1", "TP3D_SPEC_S01", "TP3D_CMR_NAIVE",
    "TP3D_CMR_LOAD_BALANCE", "TP3D_CMR_DFS", "TP3D_CMR_RANDOM_GREEDY", "TP3D_PIPE_GPIPE", "TP3D_PIPE_1F1B",
    "TP3D_PIPE_INTERLEAVED",
    "tp3d_kv_cache", "tp3d_paged_batch", "tp3d_row_strides", "kv_cache", "paged_batch", "tp3d_paged_plan",
    "tp3d_paged_store", "tp3d_paged_attn", "tp3d_paged_attn_workspace_bytes",
    "tp3d_rope", "rope", "rope_turns", "tp3d_rope_turns", "tp3d_qk_rope", "tp3d_qk_rope_bwd",
    "tp3d_qk_rope_bwd_workspace_bytes", "tp3d_paged_rope_store", "TP3D_ROPE_PLAIN", "TP3D_ROPE_LINEAR",
    "TP3D_ROPE_BASE", "TP3D_ROPE_PARTS",
    "tp3d_paged_attn_window", "tp3d_page_pool", "page_pool", "tp3d_paged_fork", "tp3d_paged_free", "tp3d_paged_compact", "tp3d_paged_copy",
]

STATUS = {0: "TP3D_OK", 1: "TP3D_EINVAL", 2: "TP3D_ESHAPE", 3: "TP3D_EALIGN", 4: "TP3D_EDTYPE",
          5: "TP3D_ECUDA", 6: "TP3D_ETIMEOUT", 7: "TP3D_EUNSUPPORTED", 8: "TP3D_EOVERLAP",
          9: "TP3D_ERANGE", 10: "TP3D_EPAGES"}
TP3D_F32, TP3D_BF16 = 0, 1
CUBE_A, CUBE_B, CUBE_C, CUBE_B_SWAP, ROW, COL, BLOCK2D, REPLICATED = range(8)
TP3D_SPEC_R, TP3D_SPEC_S0, TP3D_SPEC_S1, TP3D_SPEC_S01 = range(4)
TP3D_CMR_NAIVE, TP3D_CMR_LOAD_BALANCE, TP3D_CMR_DFS, TP3D_CMR_RANDOM_GREEDY = range(4)
TP3D_PIPE_GPIPE, TP3D_PIPE_1F1B, TP3D_PIPE_INTERLEAVED = range(3)
TP3D_SCHEME_1D, TP3D_SCHEME_2D, TP3D_SCHEME_3D = 1, 2, 3
TP3D_ROPE_PLAIN, TP3D_ROPE_LINEAR, TP3D_ROPE_BASE, TP3D_ROPE_PARTS = range(4)


class tp3d_layout(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("q", ctypes.c_int32), ("a", ctypes.c_int32), ("b", ctypes.c_int32)]


class tp3d_layer_cfg(ctypes.Structure):
    _fields_ = [("q", ctypes.c_int32), ("batch", ctypes.c_int32), ("seq", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("heads", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


PARAM_NAMES = ("ln1_g", "ln1_b", "w_qkv", "b_qkv", "w_o", "b_o", "ln2_g", "ln2_b", "w_1", "b_1", "w_2", "b_2")


class tp3d_layer_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in PARAM_NAMES]


class tp3d_layer_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in PARAM_NAMES]


class tp3d_kv_cache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page", ctypes.c_int32), ("pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p)]


class tp3d_paged_batch(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_int32), ("max_new", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("table_width", ctypes.c_int64)]


class tp3d_row_strides(ctypes.Structure):
    _fields_ = [("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class tp3d_page_pool(ctypes.Structure):
    _fields_ = [("page", ctypes.c_int32), ("rows", ctypes.c_int32), ("pages", ctypes.c_int64),
                ("table_width", ctypes.c_int64), ("free_cap", ctypes.c_int64), ("block_table", ctypes.c_void_p),
                ("shares", ctypes.c_void_p), ("free_pages", ctypes.c_void_p)]


class tp3d_rope(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("magnitude", ctypes.c_float), ("turns", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p)]
    on_host = False  # rope() was given tensors of the host, which no kernel can use


class tp3d_rect(ctypes.Structure):
    _fields_ = [("row0", ctypes.c_int64), ("rows", ctypes.c_int64), ("col0", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class tp3d_mesh_spec(ctypes.Structure):
    _fields_ = [("m1", ctypes.c_int32), ("m2", ctypes.c_int32), ("row_spec", ctypes.c_int32),
                ("col_spec", ctypes.c_int32)]


class tp3d_cmr_options(ctypes.Structure):
    _fields_ = [("algo", ctypes.c_int32), ("trials", ctypes.c_int32), ("seed", ctypes.c_uint64),
                ("node_limit", ctypes.c_int64)]


class tp3d_cmr_result(ctypes.Structure):
    _fields_ = [("makespan", ctypes.c_int64), ("nodes", ctypes.c_int64), ("complete", ctypes.c_int32),
                ("rounds", ctypes.c_int32)]


class tp3d_pipe_cfg(ctypes.Structure):
    _fields_ = [("schedule", ctypes.c_int32), ("p", ctypes.c_int32), ("m", ctypes.c_int32), ("v", ctypes.c_int32),
                ("t_f", ctypes.c_int64), ("t_b", ctypes.c_int64)]


class tp3d_pipe_op(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int32), ("microbatch", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("backward", ctypes.c_int32), ("start", ctypes.c_int64), ("end", ctypes.c_int64)]


class tp3d_pipe_result(ctypes.Structure):
    _fields_ = [("makespan", ctypes.c_int64), ("busy", ctypes.c_int64), ("idle", ctypes.c_int64),
                ("bubble", ctypes.c_double), ("max_in_flight", ctypes.c_int32)]


class Tp3dError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}" if what else STATUS.get(status, str(status)))


def check(status: int, what: str = "") -> None:
    if status != 0:
        raise Tp3dError(status, what)


def layout(kind: int, q: int = 0, a: int = 0, b: int = 0) -> tp3d_layout:
    return tp3d_layout(kind, q, a, b)


_lib = None

_SIGS = {
    "tp3d_create": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]),
    "tp3d_destroy": (None, [ctypes.c_void_p]),
    "tp3d_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "tp3d_sync_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "tp3d_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint64]),
    "tp3d_inject_load_stall": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64]),
    "tp3d_reshard": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_size_t, tp3d_layout,
                                    ctypes.c_void_p, tp3d_layout, ctypes.c_void_p, ctypes.c_void_p]),
    "tp3d_linear": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                   ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "tp3d_mlp": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tp3d_mlp_plan": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                     ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "tp3d_mlp_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    "tp3d_mlp_layout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p]),
    "tp3d_layer_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(tp3d_layer_cfg)]),
    "tp3d_layer_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_layer_cfg),
                                      ctypes.POINTER(tp3d_layer_params), ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "tp3d_layer_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_layer_cfg),
                                      ctypes.POINTER(tp3d_layer_params), ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(tp3d_layer_grads),
                                      ctypes.c_void_p]),
    "tp3d_paged_plan": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int64] +
                        [ctypes.c_void_p] * 3 + [ctypes.c_int64] + [ctypes.c_void_p] * 2 + [ctypes.c_int64] +
                        [ctypes.c_void_p] * 6),
    "tp3d_paged_store": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_kv_cache), ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p]),
    "tp3d_paged_attn": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_kv_cache),
                                       ctypes.POINTER(tp3d_paged_batch), ctypes.c_int, ctypes.c_float,
                                       ctypes.c_void_p, tp3d_row_strides, ctypes.c_void_p, tp3d_row_strides,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "tp3d_paged_attn_window": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_kv_cache),
                                              ctypes.POINTER(tp3d_paged_batch), ctypes.c_int, ctypes.c_float,
                                              ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, tp3d_row_strides,
                                              ctypes.c_void_p, tp3d_row_strides, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p]),
    "tp3d_paged_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.POINTER(tp3d_kv_cache),
                                                          ctypes.c_int]),
    "tp3d_paged_fork": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_page_pool), ctypes.c_int] +
                        [ctypes.c_void_p] * 9),
    "tp3d_paged_free": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_page_pool)] + [ctypes.c_void_p] * 5),
    "tp3d_paged_compact": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_page_pool)] + [ctypes.c_void_p] * 7),
    "tp3d_paged_copy": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_kv_cache), ctypes.c_int64] +
                        [ctypes.c_void_p] * 4),
    "tp3d_rope_turns": (ctypes.c_int, [ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double,
                                       ctypes.c_void_p, ctypes.POINTER(ctypes.c_float)]),
    "tp3d_qk_rope": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_rope), ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_int] + [ctypes.c_void_p, tp3d_row_strides] * 2 + [ctypes.c_void_p] +
                     [ctypes.c_void_p, tp3d_row_strides] * 2 + [ctypes.c_void_p]),
    "tp3d_qk_rope_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_rope), ctypes.c_int64, ctypes.c_int,
                                        ctypes.c_int] + [ctypes.c_void_p, tp3d_row_strides] * 2 + [ctypes.c_void_p] +
                         [ctypes.c_void_p, tp3d_row_strides] * 4 + [ctypes.c_void_p] * 4),
    "tp3d_qk_rope_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.POINTER(tp3d_rope)]),
    "tp3d_paged_rope_store": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_rope), ctypes.POINTER(tp3d_kv_cache),
                                             ctypes.c_int64, ctypes.c_int] + [ctypes.c_void_p, tp3d_row_strides] * 3 +
                              [ctypes.c_void_p] * 3 + [tp3d_row_strides, ctypes.c_void_p]),
    "tp3d_layout_rects": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, tp3d_layout, ctypes.POINTER(tp3d_rect),
                                         ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]),
    "tp3d_mesh_rects": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, tp3d_mesh_spec, ctypes.POINTER(tp3d_rect),
                                       ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]),
    "tp3d_cmr_plan_create": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                            ctypes.POINTER(tp3d_rect), ctypes.c_int32, ctypes.c_int32,
                                            ctypes.POINTER(tp3d_rect), ctypes.c_int32, ctypes.c_int32,
                                            ctypes.c_int32, ctypes.POINTER(ctypes.c_void_p)]),
    "tp3d_cmr_plan_destroy": (None, [ctypes.c_void_p]),
    "tp3d_cmr_plan_num_tasks": (ctypes.c_int32, [ctypes.c_void_p]),
    "tp3d_cmr_plan_task": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(tp3d_rect),
                                          ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32),
                                          ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                          ctypes.POINTER(ctypes.c_int32)]),
    "tp3d_cmr_plan_lower_bound": (ctypes.c_int64, [ctypes.c_void_p]),
    "tp3d_cmr_schedule": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(tp3d_cmr_options),
                                         ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                         ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(tp3d_cmr_result)]),
    "tp3d_pipeline_simulate": (ctypes.c_int, [ctypes.POINTER(tp3d_pipe_cfg), ctypes.POINTER(tp3d_pipe_op),
                                              ctypes.c_int64, ctypes.POINTER(tp3d_pipe_result)]),
}


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built: there is no
    fallback implementation."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m tensor_transformer_layer_cube_gb300.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def _p(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_current_raw_stream = None


def _s(stream):
    if stream is None:
        # torch's current stream as the raw handle, without building a Stream object around it
        global _current_raw_stream
        if _current_raw_stream is None:
            import torch
            torch.cuda.init()
            raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
            _current_raw_stream = lambda: raw(device())
        return _current_raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def tp3d_create(device: int = 0) -> int:
    """Returns the context handle (int); raises on failure."""
    h = ctypes.c_void_p()
    check(lib().tp3d_create(device, ctypes.byref(h)), "tp3d_create")
    return h.value


def tp3d_destroy(ctx: int) -> None:
    lib().tp3d_destroy(ctx)


def tp3d_status_string(status: int) -> str:
    return lib().tp3d_status_string(status).decode()


def tp3d_sync_status(ctx: int, stream=None) -> int:
    return lib().tp3d_sync_status(ctx, _s(stream))


def tp3d_set_wait_limit_ns(ctx: int, ns: int) -> int:
    return lib().tp3d_set_wait_limit_ns(ctx, ns)


def tp3d_inject_load_stall(ctx: int, stages: int) -> int:
    return lib().tp3d_inject_load_stall(ctx, stages)


def tp3d_reshard(ctx, R, C, elem_bytes, src_l: tp3d_layout, src, dst_l: tp3d_layout, dst, stream=None) -> int:
    return lib().tp3d_reshard(ctx, R, C, elem_bytes, src_l, _p(src), dst_l, _p(dst), _s(stream))


def tp3d_linear(ctx, q, y, M, N, K, dtype, A, B, bias, act, C, stream=None) -> int:
    return lib().tp3d_linear(ctx, q, y, M, N, K, dtype, _p(A), _p(B), _p(bias), act, _p(C), _s(stream))


def tp3d_mlp(ctx, q, M, h, f, dtype, X, W1, b1, W2, b2, Y1, Y, stream=None) -> int:
    return lib().tp3d_mlp(ctx, q, M, h, f, dtype, _p(X), _p(W1), _p(b1), _p(W2), _p(b2), _p(Y1), _p(Y), _s(stream))


def tp3d_mlp_plan(ctx, q, M, h, f):
    """(status, launches, splits): how tp3d_mlp runs a block of these sizes."""
    n, s = ctypes.c_int(0), ctypes.c_int(0)
    st = lib().tp3d_mlp_plan(ctx, q, M, h, f, ctypes.byref(n), ctypes.byref(s))
    return st, n.value, s.value


def tp3d_mlp_noalloc(ctx, q, M, h, f, dtype, X, W1, b1, W2, b2, Y, stream=None) -> int:
    """tp3d_mlp for callers that cannot allocate: the hidden activation lives
    in the library's own fixed 16 MiB device array (M * f <= 8388608)."""
    return lib().tp3d_mlp_noalloc(ctx, q, M, h, f, dtype, _p(X), _p(W1), _p(b1), _p(W2), _p(b2), _p(Y), _s(stream))


def tp3d_mlp_layout(ctx, scheme, p, M, h, f, dtype, X, W1, b1, W2, b2, Y1, Y, stream=None) -> int:
    """The MLP block in the 1-D (Megatron), 2-D (SUMMA) or 3-D (cube) layout."""
    return lib().tp3d_mlp_layout(ctx, scheme, p, M, h, f, dtype, _p(X), _p(W1), _p(b1), _p(W2), _p(b2), _p(Y1),
                                 _p(Y), _s(stream))


def tp3d_layer_workspace_bytes(cfg: tp3d_layer_cfg) -> int:
    return lib().tp3d_layer_workspace_bytes(ctypes.byref(cfg))


def _params(struct, d):
    return struct(*[_p(d.get(n)) for n in PARAM_NAMES])


def tp3d_layer_fwd(ctx, cfg: tp3d_layer_cfg, params: dict, X, Y, workspace, stream=None) -> int:
    p = _params(tp3d_layer_params, params)
    return lib().tp3d_layer_fwd(ctx, ctypes.byref(cfg), ctypes.byref(p), _p(X), _p(Y), _p(workspace), _s(stream))


def tp3d_layer_bwd(ctx, cfg: tp3d_layer_cfg, params: dict, X, workspace, dY, dX, grads: dict, stream=None) -> int:
    p = _params(tp3d_layer_params, params)
    g = _params(tp3d_layer_grads, grads)
    return lib().tp3d_layer_bwd(ctx, ctypes.byref(cfg), ctypes.byref(p), _p(X), _p(workspace), _p(dY), _p(dX),
                                ctypes.byref(g), _s(stream))


# ---------------------------------------------------------------------------
# Paged key/value cache (include/tp3d_paged.h).  Strided arguments are torch
# tensors here: their shapes and strides are what the C call takes.
# ---------------------------------------------------------------------------

_dtypes = {}
_I64, _I32 = -64, -32  # of slots and positions; no TP3D types


def _dtype_of(x):
    if not _dtypes:
        import torch
        _dtypes.update({torch.float32: TP3D_F32, torch.bfloat16: TP3D_BF16, torch.int64: _I64, torch.int32: _I32})
    return _dtypes.get(x.dtype, -1)


def kv_cache(k, v) -> tp3d_kv_cache:
    """The descriptor of two pools seen as (page, token, head, column) with
    contiguous columns (any page, token and head strides, the same for both).
    It holds their addresses: keep the tensors."""
    if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or v.dtype != k.dtype or \
            (k.stride(3) != 1 and k.shape[3] > 1):
        raise ValueError("kv_cache: two (page, token, head, column) pools of one shape, type and strides")
    return tp3d_kv_cache(_dtype_of(k), k.shape[2], k.shape[3], k.shape[1], k.shape[0], k.stride(0), k.stride(1),
                         k.stride(2), k.data_ptr(), v.data_ptr())


def paged_batch(q_start, kv_len, block_table, tokens: int, max_new: int = 0) -> tp3d_paged_batch:
    """The descriptor of one step's requests (int32 device tensors; the table
    as dense rows).  It holds their addresses: keep the tensors."""
    import torch
    for x in (q_start, kv_len, block_table):
        if x.dtype != torch.int32 or not x.is_contiguous():
            raise ValueError("paged_batch: contiguous int32 tensors")
    if block_table.dim() != 2 or block_table.shape[0] != kv_len.numel() or q_start.numel() != kv_len.numel() + 1:
        raise ValueError("paged_batch: q_start (requests + 1), kv_len (requests), block_table (requests, width)")
    return tp3d_paged_batch(kv_len.numel(), max_new, tokens, q_start.data_ptr(), kv_len.data_ptr(),
                            block_table.data_ptr(), block_table.shape[1])


def tp3d_paged_plan(ctx, page, requests, tokens, cached, fresh, free_pages, free_cap, free_count, block_table,
                    table_width, q_start, kv_len, slots, positions, free_left, stream=None) -> int:
    return lib().tp3d_paged_plan(ctx, page, requests, tokens, _p(cached), _p(fresh), _p(free_pages), free_cap,
                                 _p(free_count), _p(block_table), table_width, _p(q_start), _p(kv_len), _p(slots),
                                 _p(positions), _p(free_left), _s(stream))


def tp3d_paged_store(ctx, cache: tp3d_kv_cache, K, V, slots, stream=None) -> int:
    """K, V: (token, head, column) tensors of the same strides."""
    shape, st = K.shape, K.stride()
    if len(shape) != 3 or st[2] != 1 or V.shape != shape or V.stride() != st or shape[1] != cache.kv_heads or \
            shape[2] != cache.head_dim:
        raise ValueError("tp3d_paged_store: K and V (tokens, kv_heads, head_dim) of the same strides, "
                         "contiguous columns")
    dt = cache.dtype
    if _dtype_of(K) != dt or _dtype_of(V) != dt or slots.numel() < shape[0] or _dtype_of(slots) != _I64 or \
            not slots.is_contiguous():
        raise ValueError("tp3d_paged_store: K and V of the cache's type, an int64 slot for each token")
    return lib().tp3d_paged_store(ctx, ctypes.byref(cache), shape[0], K.data_ptr(), V.data_ptr(), st[0], st[1],
                                  slots.data_ptr(), _s(stream))


def tp3d_paged_attn(ctx, cache: tp3d_kv_cache, batch: tp3d_paged_batch, Q, O, lse, scale, workspace,
                    stream=None) -> int:
    """Q, O: (token, head, column) tensors; lse: dense (token, head) float32 or None."""
    heads, rows = _attn_rows("tp3d_paged_attn", cache, batch, Q, O, lse)
    return lib().tp3d_paged_attn(ctx, cache, batch, heads, scale, *rows, _p(lse),
                                 _p(workspace), _s(stream))


def tp3d_paged_attn_window(ctx, cache: tp3d_kv_cache, batch: tp3d_paged_batch, Q, O, lse, scale, window, sinks,
                           workspace, stream=None) -> int:
    """tp3d_paged_attn over a sliding window of ``window`` keys and the first ``sinks`` ones."""
    heads, rows = _attn_rows("tp3d_paged_attn_window", cache, batch, Q, O, lse)
    return lib().tp3d_paged_attn_window(ctx, cache, batch, heads, scale, window, sinks,
                                        *rows, _p(lse), _p(workspace), _s(stream))


def _attn_rows(what, cache, batch, Q, O, lse):
    shape, qs, os_ = Q.shape, Q.stride(), O.stride()
    dt = cache.dtype
    if len(shape) != 3 or O.shape != shape or qs[2] != 1 or os_[2] != 1 or shape[0] < batch.tokens or \
            shape[2] != cache.head_dim or _dtype_of(Q) != dt or _dtype_of(O) != dt:
        raise ValueError(f"{what}: Q and O (tokens, heads, head_dim) of the cache's type, contiguous columns")
    if lse is not None and (not lse.is_contiguous() or lse.shape != shape[:2] or _dtype_of(lse) != TP3D_F32):
        raise ValueError(f"{what}: lse dense (tokens, heads) float32")
    return shape[1], (Q.data_ptr(), _strides_of(Q), O.data_ptr(), _strides_of(O))


def tp3d_paged_attn_workspace_bytes(ctx, cache: tp3d_kv_cache, heads: int) -> int:
    return lib().tp3d_paged_attn_workspace_bytes(ctx, ctypes.byref(cache), heads)


def page_pool(page: int, block_table, shares, free_pages) -> tp3d_page_pool:
    """The descriptor of a pool's bookkeeping (int32 device tensors; the table as dense rows, one share count for each
    page).  It holds their addresses: keep the tensors."""
    if block_table.dim() != 2 or shares.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("page_pool: block_table (rows, width), shares (pages), free_pages (entries)")
    _words("page_pool", (0, 0, 0), block_table, shares, free_pages)
    return tp3d_page_pool(page, block_table.shape[0], shares.numel(), block_table.shape[1], free_pages.numel(),
                          block_table.data_ptr(), shares.data_ptr(), free_pages.data_ptr())


_int32 = None


def _words(what, sizes, *arrays):
    """Pointers of contiguous int32 tensors of at least so many elements each."""
    global _int32
    if _int32 is None:
        import torch
        _int32 = torch.int32
    out = []
    for n, x in zip(sizes, arrays):
        if x.dtype is not _int32 or x.numel() < n or not x.is_contiguous():
            raise ValueError(f"{what}: contiguous int32 tensors, one element for each of what they describe")
        out.append(x.data_ptr())
    return out


def tp3d_paged_fork(ctx, pool: tp3d_page_pool, src, dst, len, free_count, free_left, copy_from, copy_to, copy_count,
                    stream=None) -> int:
    """One fork for each element of ``src``."""
    n = src.numel()
    return lib().tp3d_paged_fork(ctx, pool, n,
                                 *_words("tp3d_paged_fork", (n, n, n, 1, 1, n, n, 1), src, dst, len, free_count,
                                         free_left, copy_from, copy_to, copy_count), _s(stream))


def tp3d_paged_free(ctx, pool: tp3d_page_pool, first, end, free_count, free_left, stream=None) -> int:
    n = pool.rows
    return lib().tp3d_paged_free(ctx, pool, *_words("tp3d_paged_free", (n, n, 1, 1), first, end, free_count, free_left),
                                 _s(stream))


def tp3d_paged_compact(ctx, pool: tp3d_page_pool, kv_len, free_count, page_map, copy_from, copy_to, copy_count,
                       stream=None) -> int:
    n = pool.pages
    return lib().tp3d_paged_compact(ctx, pool,
                                    *_words("tp3d_paged_compact", (pool.rows, 1, n, n // 2, n // 2, 1), kv_len,
                                            free_count, page_map, copy_from, copy_to, copy_count), _s(stream))


def tp3d_paged_copy(ctx, cache: tp3d_kv_cache, copies: int, copy_from, copy_to, copy_count=None, stream=None) -> int:
    at, to = _words("tp3d_paged_copy", (copies, copies), copy_from, copy_to)
    count = None if copy_count is None else _words("tp3d_paged_copy", (1,), copy_count)[0]
    return lib().tp3d_paged_copy(ctx, cache, copies, at, to, count, _s(stream))


# ---------------------------------------------------------------------------
# Head norms with the rotation by position (include/tp3d_rope.h).
# ---------------------------------------------------------------------------

def tp3d_rope_turns(rotary_dim, base, kind, factor, context, turns) -> tuple:
    """(status, magnitude); ``turns``: a host tensor of int64 words, rotary_dim / 2 of them, or None."""
    if turns is not None and (_dtype_of(turns) != _I64 or turns.device.type != "cpu" or not turns.is_contiguous() or
                              turns.numel() < rotary_dim // 2):
        raise ValueError("tp3d_rope_turns: rotary_dim / 2 contiguous int64 words in host memory")
    m = ctypes.c_float(0.0)
    st = lib().tp3d_rope_turns(rotary_dim, base, kind, factor, context, _p(turns), ctypes.byref(m))
    return st, m.value


def rope_turns(rotary_dim: int, base: float = 10000.0, kind: int = TP3D_ROPE_PLAIN, factor: float = 1.0,
               context: float = 1.0) -> tuple:
    """(turns, magnitude): the frequencies as a host tensor of int64 words, for ``rope`` once it is on the device.
    Raises on failure."""
    import torch
    turns = torch.empty(max(rotary_dim, 0) // 2, dtype=torch.int64)
    st, magnitude = tp3d_rope_turns(rotary_dim, base, kind, factor, context, turns)
    check(st, "tp3d_rope_turns")
    return turns, magnitude


def rope(turns, dtype, head_dim: int, rotary_dim: int, interleaved: bool = False, magnitude: float = 1.0,
         norm: bool = False, eps: float = 1e-6, q_weight=None, k_weight=None) -> tp3d_rope:
    """The descriptor of a norm and rotation of heads of ``dtype`` (a torch dtype): device tensors, the frequencies
    int64 words.  It holds their addresses: keep the tensors."""
    import torch
    code = {torch.float32: TP3D_F32, torch.bfloat16: TP3D_BF16}.get(dtype)
    if code is None:
        raise ValueError("rope: heads of bfloat16 or float32")
    if rotary_dim and (turns is None or turns.dtype != torch.int64 or not turns.is_contiguous() or
                       turns.numel() < rotary_dim // 2):
        raise ValueError("rope: rotary_dim / 2 contiguous int64 words of turns")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype != dtype or not w.is_contiguous() or w.numel() != head_dim):
            raise ValueError("rope: weights of head_dim contiguous elements of the heads' type")
    r = tp3d_rope(code, head_dim, rotary_dim, int(interleaved), int(norm), eps, magnitude, _p(turns), _p(q_weight),
                  _p(k_weight))
    used = ([turns] if rotary_dim else []) + ([q_weight, k_weight] if norm else [])
    r.on_host = any(x is not None and not x.is_cuda for x in used)
    return r


def _on_device(what, rope):
    """Last of a call's checks: the descriptor's tensors, of which the kernels get the addresses."""
    if rope.on_host:
        raise TypeError(f"{what}: turns and weights in device memory (rope_turns makes a host tensor)")


_row_strides = {}  # by a tensor's strides


def _strides_of(x):
    """The token and head strides of a (token, head, column) tensor; None where columns are not contiguous."""
    st = x.stride()
    r = _row_strides.get(st)
    if r is None:
        if len(st) != 3 or st[2] != 1:
            return None
        if len(_row_strides) > 1000:
            _row_strides.clear()
        r = _row_strides[st] = tp3d_row_strides(st[0], st[1])
    return r


def _rows_of(what, r: tp3d_rope, shape, a, b):
    """Pointers and strides of two (token, head, column) tensors of one shape, checked."""
    sa, sb, dt = _row_strides.get(a.stride()) or _strides_of(a), _row_strides.get(b.stride()) or _strides_of(b), r.dtype
    if len(shape) != 3 or shape[2] != r.head_dim or sa is None or sb is None or a.shape != shape or b.shape != shape or \
            _dtype_of(a) != dt or _dtype_of(b) != dt:
        raise ValueError(f"{what}: (tokens, heads, head_dim) rows of one type, contiguous columns, the same heads for what "
                         "belongs together")
    return a.data_ptr(), sa, b.data_ptr(), sb


def _positions(what, positions, tokens):
    if _dtype_of(positions) != _I32 or positions.numel() < tokens or not positions.is_contiguous():
        raise ValueError(f"{what}: a contiguous int32 position for each token")
    return positions.data_ptr()


def tp3d_qk_rope(ctx, rope: tp3d_rope, Q, K, positions, Q_out, K_out, stream=None) -> int:
    """Q, Q_out (tokens, heads, head_dim), K, K_out (tokens, kv_heads, head_dim); in place where the same tensor."""
    what, qs, ks = "tp3d_qk_rope", Q.shape, K.shape
    q, qst, qo, qost = _rows_of(what, rope, qs, Q, Q_out)
    k, kst, ko, kost = _rows_of(what, rope, ks, K, K_out)
    n = qs[0]
    if ks[0] != n:
        raise ValueError("tp3d_qk_rope: Q and K of the same tokens")
    at = _positions(what, positions, n)
    _on_device(what, rope)
    return lib().tp3d_qk_rope(ctx, rope, n, qs[1], ks[1], q, qst, k, kst, at, qo, qost, ko, kost, _s(stream))


def tp3d_qk_rope_bwd(ctx, rope: tp3d_rope, Q, K, positions, dQ_out, dK_out, dQ, dK, dq_weight, dk_weight, workspace,
                     stream=None) -> int:
    """Shapes as in tp3d_qk_rope; Q and K may be None without the norm.  dq_weight, dk_weight: head_dim elements or
    None."""
    what, qs, ks = "tp3d_qk_rope_bwd", dQ_out.shape, dK_out.shape
    none = (None, _no_strides)
    q, qst = _rows_of(what, rope, qs, Q, Q)[:2] if Q is not None else none
    k, kst = _rows_of(what, rope, ks, K, K)[:2] if K is not None else none
    gq, gqst, dq, dqst = _rows_of(what, rope, qs, dQ_out, dQ)
    gk, gkst, dk, dkst = _rows_of(what, rope, ks, dK_out, dK)
    n = qs[0]
    if ks[0] != n:
        raise ValueError("tp3d_qk_rope_bwd: Q and K of the same tokens")
    for w in (dq_weight, dk_weight):
        if w is not None and (_dtype_of(w) != rope.dtype or not w.is_contiguous() or w.numel() != rope.head_dim):
            raise ValueError("tp3d_qk_rope_bwd: weights' gradients of head_dim contiguous elements of the heads' type")
    at = _positions(what, positions, n)
    _on_device(what, rope)
    return lib().tp3d_qk_rope_bwd(ctx, rope, n, qs[1], ks[1], q, qst, k, kst, at, gq, gqst, gk, gkst, dq, dqst, dk, dkst,
                                  _p(dq_weight), _p(dk_weight), _p(workspace), _s(stream))


_no_strides = tp3d_row_strides(0, 0)


def tp3d_qk_rope_bwd_workspace_bytes(ctx, rope: tp3d_rope) -> int:
    return lib().tp3d_qk_rope_bwd_workspace_bytes(ctx, ctypes.byref(rope))


def tp3d_paged_rope_store(ctx, rope: tp3d_rope, cache: tp3d_kv_cache, Q, K, V, positions, slots, Q_out,
                          stream=None) -> int:
    """Q, Q_out (tokens, heads, head_dim), K, V (tokens, kv_heads, head_dim); an int64 slot for each token."""
    what, qs, ks = "tp3d_paged_rope_store", Q.shape, K.shape
    q, qst, qo, qost = _rows_of(what, rope, qs, Q, Q_out)
    k, kst, v, vst = _rows_of(what, rope, ks, K, V)
    n = qs[0]
    if ks[0] != n or ks[1] != cache.kv_heads:
        raise ValueError("tp3d_paged_rope_store: K and V of Q's tokens and the cache's heads")
    if _dtype_of(slots) != _I64 or slots.numel() < n or not slots.is_contiguous():
        raise ValueError("tp3d_paged_rope_store: an int64 slot for each token")
    at = _positions(what, positions, n)
    _on_device(what, rope)
    return lib().tp3d_paged_rope_store(ctx, rope, cache, n, qs[1], q, qst, k, kst, v, vst, at, slots.data_ptr(), qo, qost,
                                       _s(stream))


# ---------------------------------------------------------------------------
# Host-side planners (include/tp3d_plan.h): no GPU involved.  Rectangles are
# (row0, rows, col0, cols) tuples.
# ---------------------------------------------------------------------------

def _rects_out(fn, R, C, spec):
    n = ctypes.c_int32(0)
    st = fn(R, C, spec, None, 0, ctypes.byref(n))
    if n.value <= 0:
        return st, []
    arr = (tp3d_rect * n.value)()
    st = fn(R, C, spec, arr, n.value, ctypes.byref(n))
    return st, [(r.row0, r.rows, r.col0, r.cols) for r in arr] if st == 0 else []


def tp3d_layout_rects(R, C, l: tp3d_layout):
    """(status, rectangles of the layout's shards in shard order)."""
    return _rects_out(lib().tp3d_layout_rects, R, C, l)


def tp3d_mesh_rects(R, C, s: tp3d_mesh_spec):
    """(status, rectangles of the mesh devices in mesh order)."""
    return _rects_out(lib().tp3d_mesh_rects, R, C, s)


def _rect_array(rects):
    arr = (tp3d_rect * len(rects))()
    for k, r in enumerate(rects):
        arr[k] = tp3d_rect(*r)
    return arr


def tp3d_cmr_plan_create(R, C, elem_bytes, src_rects, src_first, dst_rects, dst_first, devices_per_host):
    """(status, plan handle or None)."""
    h = ctypes.c_void_p()
    st = lib().tp3d_cmr_plan_create(R, C, elem_bytes, _rect_array(src_rects), len(src_rects), src_first,
                                    _rect_array(dst_rects), len(dst_rects), dst_first, devices_per_host,
                                    ctypes.byref(h))
    return st, h.value


def tp3d_cmr_plan_destroy(plan) -> None:
    lib().tp3d_cmr_plan_destroy(plan)


def tp3d_cmr_plan_num_tasks(plan) -> int:
    return lib().tp3d_cmr_plan_num_tasks(plan)


def tp3d_cmr_plan_task(plan, i, max_senders, max_receivers):
    """(status, slice, duration, sender devices, receiver devices) of task i;
    max_senders / max_receivers: the create call's source / destination
    device counts."""
    r, d = tp3d_rect(), ctypes.c_int64()
    ns, nr = ctypes.c_int32(), ctypes.c_int32()
    sa, ra = (ctypes.c_int32 * max_senders)(), (ctypes.c_int32 * max_receivers)()
    st = lib().tp3d_cmr_plan_task(plan, i, ctypes.byref(r), ctypes.byref(d), sa, ctypes.byref(ns), ra,
                                  ctypes.byref(nr))
    if st != 0:
        return st, None, None, [], []
    return st, (r.row0, r.rows, r.col0, r.cols), d.value, list(sa[:ns.value]), list(ra[:nr.value])


def tp3d_cmr_plan_lower_bound(plan) -> int:
    return lib().tp3d_cmr_plan_lower_bound(plan)


def tp3d_cmr_schedule(plan, algo, trials=1, seed=0, node_limit=1):
    """(status, sender host per task, global order, start time per task,
    tp3d_cmr_result)."""
    n = max(lib().tp3d_cmr_plan_num_tasks(plan), 0)
    snd, order, start = (ctypes.c_int32 * n)(), (ctypes.c_int32 * n)(), (ctypes.c_int64 * n)()
    res = tp3d_cmr_result()
    opt = tp3d_cmr_options(algo, trials, seed, node_limit)
    st = lib().tp3d_cmr_schedule(plan, ctypes.byref(opt), snd, order, start, ctypes.byref(res))
    return st, list(snd), list(order), list(start), res


def tp3d_pipeline_simulate(cfg: tp3d_pipe_cfg, want_ops: bool = False):
    """(status, tp3d_pipe_result, list of tp3d_pipe_op or None)."""
    res = tp3d_pipe_result()
    if not want_ops:
        return lib().tp3d_pipeline_simulate(ctypes.byref(cfg), None, 0, ctypes.byref(res)), res, None
    n = 2 * max(cfg.p, 0) * max(cfg.m, 0) * max(cfg.v, 0)
    ops = (tp3d_pipe_op * max(n, 1))()
    st = lib().tp3d_pipeline_simulate(ctypes.byref(cfg), ops, n, ctypes.byref(res))
    return st, res, list(ops[:n]) if st == 0 else None
