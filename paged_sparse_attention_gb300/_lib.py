"""ctypes binding of liboomb.so: argument marshalling only.

Every function here forwards to the C entry point of the same name in
include/oomb.h, passing raw device pointers taken from torch tensors.  There is
no fallback: if liboomb.so is missing the import of the binding fails loudly.
"""
from __future__ import annotations

import ctypes as C
import os
import re
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "liboomb.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "oomb.h")

OOMB_BF16, OOMB_FP32 = 0, 1
OOMB_CTRL_WORDS = 16  # uint32 words of a pool's control block (error bits + selection barrier state)
OOMB_OP_SELECT, OOMB_OP_BWD, OOMB_OP_SCORE_FWD, OOMB_OP_SCORE_BWD = 0, 1, 2, 3
STATUS = {0: "OK", 1: "ERR_ARG", 2: "ERR_OUT_OF_PAGES", 3: "ERR_ALIGN", 4: "ERR_DTYPE", 5: "ERR_KERNEL",
          6: "ERR_TIMEOUT", 7: "ERR_CUDA", 8: "ERR_UNSUPPORTED", 9: "ERR_WORKSPACE"}


class OombError(RuntimeError):
    def __init__(self, func: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{func}: {STATUS.get(status, status)} ({detail})")


class PoolDesc(C.Structure):
    _fields_ = [
        ("n_q_heads", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("page_size", C.c_int),
        ("num_phys_pages", C.c_int), ("max_logical_pages", C.c_int), ("dtype", C.c_int),
        ("k_pool", C.c_void_p), ("v_pool", C.c_void_p), ("dk_pool", C.c_void_p), ("dv_pool", C.c_void_p),
        ("summary", C.c_void_p), ("page_table", C.c_void_p), ("error_word", C.c_void_p),
        ("page_order", C.c_void_p), ("offload", C.c_int), ("stage_k", C.c_void_p), ("stage_v", C.c_void_p),
        ("stage_max_sel", C.c_int), ("offload_grads", C.c_int), ("stage_dk", C.c_void_p),
        ("stage_dv", C.c_void_p), ("grad_state", C.c_void_p),
    ]


class ScoreMod(C.Structure):
    _fields_ = [("softcap", C.c_float), ("slopes", C.c_void_p), ("key_begin", C.c_void_p), ("key_end", C.c_void_p)]


_lib: Optional[C.CDLL] = None


def header_symbols():
    """Names of the entry points include/oomb.h declares."""
    with open(HEADER) as f:
        txt = f.read()
    return sorted(set(re.findall(r"OOMB_API\s+[\w\s\*]+?\b(oomb_\w+)\s*\(", txt)))


def load(path: str = LIB_PATH) -> C.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run __graft_entry__.build() (nvcc, sm_103a)")
    lib = C.CDLL(path)
    vp, i32, i64, f32, sz = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t
    sig = {
        "oomb_pool_create": (i32, [C.POINTER(PoolDesc), C.POINTER(vp)]),
        "oomb_pool_destroy": (None, [vp]),
        "oomb_pool_reset": (i32, [vp, vp]),
        "oomb_kv_append": (i32, [vp, vp, vp, i64, i32, vp]),
        "oomb_kv_append_staged": (i32, [vp, vp, vp, i64, i32, vp, i32, i32, vp]),
        "oomb_kv_append_deferred": (i32, [vp, vp, vp, i64, i32, vp, i32, i32, vp]),
        "oomb_page_select_append": (i32, [vp, vp, vp, vp, i64, i32, i32, i32, vp, vp, i32, vp, sz, i32, i32, vp]),
        "oomb_kv_writeback": (i32, [vp, vp, vp, i32, i32, i64, i64, vp]),
        "oomb_page_select": (i32, [vp, vp, i64, i32, i32, i32, vp, vp, i32, vp, sz, vp]),
        "oomb_chunk_attn_fwd": (i32, [vp, vp, i64, i32, vp, vp, i32, f32, vp, vp, vp]),
        "oomb_chunk_attn_bwd": (i32, [vp, vp, vp, vp, vp, i64, i32, vp, vp, i32, f32, vp, vp, sz, vp]),
        "oomb_score_attn_fwd": (i32, [vp, vp, i64, i32, vp, vp, i32, f32, C.POINTER(ScoreMod), vp, vp, vp, sz, vp]),
        "oomb_score_attn_bwd": (i32, [vp, vp, vp, vp, vp, i64, i32, vp, vp, i32, f32, C.POINTER(ScoreMod), vp, vp, sz,
                                      vp]),
        "oomb_doc_spans": (i32, [vp, vp, i32, i64, i32, vp, vp, vp]),
        "oomb_prefetch": (i32, [vp, vp, vp, i32, i32, vp]),
        "oomb_pool_set_stage": (i32, [vp, i32]),
        "oomb_prefetch_pages": (i32, [vp, vp, vp, i32, i32, i64, i64, vp]),
        "oomb_gemm": (i32, [i32, i32, i32, i32, i32, vp, vp, vp, i32, i32, f32, f32, vp, sz, vp]),
        "oomb_bias_rope": (i32, [vp, i32, vp, vp, i32, i32, i32, i32, i64, f32, i32, vp]),
        "oomb_bias_rope_axes": (i32, [vp, i32, vp, vp, i32, i32, i32, i32, vp, i32, vp, f32, i32, i32, vp]),
        "oomb_block_norm_fwd": (i32, [vp, vp, vp, vp, i32, vp, f32, f32, i32, i32, i32, vp, vp, vp, vp, vp]),
        "oomb_block_norm_bwd": (i32, [vp, vp, vp, vp, i32, vp, f32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                      i32, vp, sz, vp]),
        "oomb_block_norm_workspace": (sz, [i32, i32]),
        "oomb_block_norm_check": (i32, [vp, C.POINTER(C.c_uint32)]),
        "oomb_block_norm_test_timeout": (None, [i32]),
        "oomb_embed_fwd": (i32, [vp, i32, vp, i32, i32, i32, f32, vp, vp, vp]),
        "oomb_embed_bwd": (i32, [vp, i32, vp, i32, i32, i32, f32, vp, i32, vp, sz, vp, vp]),
        "oomb_embed_workspace": (sz, [i32, i32]),
        "oomb_layer_norm_fwd": (i32, [vp, vp, vp, f32, i32, i32, i32, vp, vp, vp, vp]),
        "oomb_layer_norm_bwd": (i32, [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, i32, vp, sz, vp]),
        "oomb_layer_norm_workspace": (sz, [i32, i32]),
        "oomb_head_loss_fwd": (i32, [vp, vp, vp, i32, i32, i32, i32, f32, vp, vp, vp, sz, vp, vp]),
        "oomb_head_loss_bwd": (i32, [vp, vp, vp, vp, vp, f32, i32, i32, i32, i32, f32, vp, vp, i32, i32, vp, sz, vp,
                                     vp]),
        "oomb_head_loss_workspace": (sz, [i32, i32, i32, i32, i32]),
        "oomb_word_check": (i32, [vp, vp, C.POINTER(C.c_uint32)]),
        "oomb_grad_gather": (i32, [vp, i64, i32, vp, vp, vp]),
        "oomb_grad_prefetch": (i32, [vp, vp, vp, i32, vp, vp, i32, vp]),
        "oomb_grad_carry": (i32, [vp, vp, vp, i32, vp, vp, i32, vp]),
        "oomb_grad_writeback": (i32, [vp, vp, vp, i32, i32, vp]),
        "oomb_workspace_size": (sz, [vp, i32, i32]),
        "oomb_check": (i32, [vp, vp, C.POINTER(C.c_uint32)]),
        "oomb_page_table_host": (i32, [vp, vp, i32]),
        "oomb_pool_tokens": (i64, [vp]),
        "oomb_pool_free_pages": (i32, [vp]),
        "oomb_status_str": (C.c_char_p, [i32]),
        "oomb_uses_tensor_cores": (i32, [vp]),
        "oomb_launch_count": (C.c_uint64, []),
        "oomb_page_select_noalloc": (i32, [vp, vp, i64, i32, i32, i32, vp, vp, i32, vp]),
        "oomb_window_select": (i32, [vp, i64, i32, i32, i32, vp, vp, i32, vp]),
        "oomb_page_free": (i32, [vp, i64, i32, vp]),
        "oomb_last_cuda_error": (C.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr() if hasattr(t, "data_ptr") else int(t)


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # a Stream object costs microseconds
        return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ok(name: str, st: int):
    if st != 0:
        detail = load().oomb_status_str(st).decode()
        if st == 7:
            detail += ": " + load().oomb_last_cuda_error().decode()
        raise OombError(name, st, detail)


# Head layout and dtype of the live pools, by handle: what the tensors of the calls below
# that take a pool and check their tensors are checked against.
_pools = {}


def _need(func: str, name: str, t, shape, dtype, dev: int) -> int:
    """Address of a tensor that a kernel reads or writes as it is: on CUDA device ``dev``,
    contiguous, of this shape and dtype.  Anything else is refused."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{func}: {name} is missing")
    if t.dtype is not dtype:
        raise TypeError(f"{func}: {name} has to be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{func}: {name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{func}: {name} is on {t.device}, not on the current CUDA device")
    raise ValueError(f"{func}: {name} is not contiguous")


def _opt(func: str, name: str, t, shape, dtype, dev: int) -> Optional[int]:
    return None if t is None else _need(func, name, t, shape, dtype, dev)


def _dims(func: str, name: str, t, n: int):
    """Shape of a tensor that sets the sizes the others are checked against."""
    if t is None or t.dim() != n:
        raise ValueError(f"{func}: {name} has to have {n} dimensions")
    return t.shape


def _scratch(func: str, t, dev: int):
    """Address and bytes of a workspace (None: no bytes)."""
    if t is None:
        return None, 0
    return _need(func, "workspace", t, t.shape, t.dtype, dev), t.numel() * t.element_size()


# ---------------------------------------------------------------- entry points
def oomb_pool_create(desc: PoolDesc) -> int:
    h = C.c_void_p()
    _ok("oomb_pool_create", load().oomb_pool_create(C.byref(desc), C.byref(h)))
    _pools[h.value] = (desc.n_q_heads, desc.n_kv_heads, desc.head_dim, desc.dtype)
    return h.value


def oomb_pool_destroy(pool: int) -> None:
    _pools.pop(pool, None)
    load().oomb_pool_destroy(pool)


def oomb_pool_reset(pool: int, stream=None) -> None:
    _ok("oomb_pool_reset", load().oomb_pool_reset(pool, _stream(stream)))


def oomb_kv_append(pool: int, k, v, first_token: int, n_tokens: Optional[int] = None, stream=None) -> None:
    n = k.shape[0] if n_tokens is None else n_tokens
    _ok("oomb_kv_append", load().oomb_kv_append(pool, _ptr(k), _ptr(v), first_token, n, _stream(stream)))


def oomb_kv_append_staged(pool: int, k, v, first_token: int, sel_count, max_sel: int, stage_buf: int,
                          n_tokens: Optional[int] = None, stream=None) -> None:
    n = k.shape[0] if n_tokens is None else n_tokens
    _ok("oomb_kv_append_staged", load().oomb_kv_append_staged(pool, _ptr(k), _ptr(v), first_token, n, _ptr(sel_count),
                                                              max_sel, stage_buf, _stream(stream)))


def oomb_kv_append_deferred(pool: int, k, v, first_token: int, sel_count, max_sel: int, stage_buf: int,
                            n_tokens: Optional[int] = None, stream=None) -> None:
    n = k.shape[0] if n_tokens is None else n_tokens
    _ok("oomb_kv_append_deferred", load().oomb_kv_append_deferred(pool, _ptr(k), _ptr(v), first_token, n,
                                                                  _ptr(sel_count), max_sel, stage_buf, _stream(stream)))


def oomb_kv_writeback(pool: int, sel, sel_count, stage_buf: int, first_page: int, end_page: int,
                      stream=None) -> None:
    _ok("oomb_kv_writeback", load().oomb_kv_writeback(pool, _ptr(sel), _ptr(sel_count), sel.shape[-1], stage_buf,
                                                      first_page, end_page, _stream(stream)))


def oomb_page_select(pool: int, q, q_start: int, top_k: int, n_sink: int, sel, sel_count, workspace,
                     n_q: Optional[int] = None, stream=None) -> None:
    n = q.shape[0] if n_q is None else n_q
    ws_bytes = workspace.numel() * workspace.element_size()
    _ok("oomb_page_select", load().oomb_page_select(pool, _ptr(q), q_start, n, top_k, n_sink, _ptr(sel),
                                                    _ptr(sel_count), sel.shape[-1], _ptr(workspace), ws_bytes,
                                                    _stream(stream)))


def oomb_page_free(pool: int, first_logical_page: int, n_pages: int, stream=None) -> None:
    _ok("oomb_page_free", load().oomb_page_free(pool, first_logical_page, n_pages, _stream(stream)))


def oomb_window_select(pool: int, q_start: int, n_q: int, window: int, n_sink: int, sel, sel_count,
                       stream=None) -> None:
    _ok("oomb_window_select", load().oomb_window_select(pool, q_start, n_q, window, n_sink, _ptr(sel),
                                                        _ptr(sel_count), sel.shape[-1], _stream(stream)))


def oomb_chunk_attn_fwd(pool: int, q, q_start: int, sel, sel_count, softmax_scale: float, o, lse,
                        n_q: Optional[int] = None, stream=None) -> None:
    n = q.shape[0] if n_q is None else n_q
    _ok("oomb_chunk_attn_fwd", load().oomb_chunk_attn_fwd(pool, _ptr(q), q_start, n, _ptr(sel), _ptr(sel_count),
                                                          sel.shape[-1], softmax_scale, _ptr(o), _ptr(lse),
                                                          _stream(stream)))


def oomb_chunk_attn_bwd(pool: int, q, o, d_o, lse, q_start: int, sel, sel_count, softmax_scale: float, dq,
                        workspace, n_q: Optional[int] = None, stream=None) -> None:
    n = q.shape[0] if n_q is None else n_q
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _ok("oomb_chunk_attn_bwd", load().oomb_chunk_attn_bwd(pool, _ptr(q), _ptr(o), _ptr(d_o), _ptr(lse), q_start, n,
                                                          _ptr(sel), _ptr(sel_count), sel.shape[-1], softmax_scale,
                                                          _ptr(dq), _ptr(workspace), ws_bytes, _stream(stream)))


def _score_call(func: str, pool: int, q, rows, lse, sel, sel_count, workspace, softcap, slopes, key_begin, key_end):
    """Checks the tensors of a score_attn call; (n_q, max_sel, ScoreMod, addresses by name)."""
    import torch
    if pool not in _pools:
        raise ValueError(f"{func}: not a live pool")
    Hq, Hkv, d, code = _pools[pool]
    dt, i32, f32, i64 = (torch.float32 if code == OOMB_FP32 else torch.bfloat16), torch.int32, torch.float32, torch.int64
    dev = torch.cuda.current_device()
    n = _dims(func, "q", q, 3)[0]
    shape = (n, Hq, d)
    at = {"q": _need(func, "q", q, shape, dt, dev)}
    for name, t in rows.items():
        at[name] = _need(func, name, t, shape, dt, dev)
    at["lse"] = _need(func, "lse", lse, (Hq, n), f32, dev)
    max_sel = _dims(func, "sel", sel, 2)[1]
    at["sel"] = _need(func, "sel", sel, (Hkv, max_sel), i32, dev)
    at["sel_count"] = _need(func, "sel_count", sel_count, (Hkv,), i32, dev)
    mod = ScoreMod(softcap, _opt(func, "slopes", slopes, (Hq,), f32, dev),
                   _opt(func, "key_begin", key_begin, (n,), i64, dev), _opt(func, "key_end", key_end, (n,), i64, dev))
    at["ws"], at["ws_bytes"] = _scratch(func, workspace, dev)
    return n, max_sel, mod, at


def oomb_score_attn_fwd(pool: int, q, q_start: int, sel, sel_count, softmax_scale: float, o, lse, workspace=None,
                        softcap: float = 0.0, slopes=None, key_begin=None, key_end=None, stream=None) -> None:
    """oomb_chunk_attn_fwd with capped scores, a distance bias and per-row key ranges."""
    n, max_sel, mod, at = _score_call("oomb_score_attn_fwd", pool, q, {"o": o}, lse, sel, sel_count, workspace, softcap,
                                      slopes, key_begin, key_end)
    _ok("oomb_score_attn_fwd", load().oomb_score_attn_fwd(pool, at["q"], q_start, n, at["sel"], at["sel_count"], max_sel,
                                                          softmax_scale, C.byref(mod), at["o"], at["lse"], at["ws"],
                                                          at["ws_bytes"], _stream(stream)))


def oomb_score_attn_bwd(pool: int, q, o, d_o, lse, q_start: int, sel, sel_count, softmax_scale: float, dq, workspace,
                        softcap: float = 0.0, slopes=None, key_begin=None, key_end=None, stream=None) -> None:
    """The backward of oomb_score_attn_fwd: dq written, dK/dV added into the gradient pools."""
    n, max_sel, mod, at = _score_call("oomb_score_attn_bwd", pool, q, {"o": o, "d_o": d_o, "dq": dq}, lse, sel,
                                      sel_count, workspace, softcap, slopes, key_begin, key_end)
    _ok("oomb_score_attn_bwd", load().oomb_score_attn_bwd(pool, at["q"], at["o"], at["d_o"], at["lse"], q_start, n,
                                                          at["sel"], at["sel_count"], max_sel, softmax_scale,
                                                          C.byref(mod), at["dq"], at["ws"], at["ws_bytes"],
                                                          _stream(stream)))


def oomb_doc_spans(doc_start, q_start: int, key_begin, key_end, prefix_len=None, stream=None) -> None:
    """Key ranges of packed documents (boundaries doc_start [n_docs + 1], optional prefix_len [n_docs])."""
    import torch
    f, dev, i64 = "oomb_doc_spans", torch.cuda.current_device(), torch.int64
    n_docs = _dims(f, "doc_start", doc_start, 1)[0] - 1
    n = _dims(f, "key_begin", key_begin, 1)[0]
    _ok(f, load().oomb_doc_spans(_need(f, "doc_start", doc_start, (n_docs + 1,), i64, dev),
                                 _opt(f, "prefix_len", prefix_len, (n_docs,), i64, dev), n_docs, q_start, n,
                                 _need(f, "key_begin", key_begin, (n,), i64, dev),
                                 _need(f, "key_end", key_end, (n,), i64, dev), _stream(stream)))


def oomb_prefetch(pool: int, sel, sel_count, stage_buf: int, stream=None) -> None:
    _ok("oomb_prefetch", load().oomb_prefetch(pool, _ptr(sel), _ptr(sel_count), sel.shape[-1], stage_buf,
                                              _stream(stream)))


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return OOMB_FP32
    if t.dtype == torch.bfloat16:
        return OOMB_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def oomb_gemm(a, b, c, trans_a: bool = False, trans_b: bool = False, alpha: float = 1.0, beta: float = 0.0,
              workspace=None, stream=None) -> None:
    """c[m, n] = alpha op(a) op(b) + beta c (row-major, contiguous tensors)."""
    m, n = c.shape
    k = a.shape[0] if trans_a else a.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _ok("oomb_gemm", load().oomb_gemm(m, n, k, int(trans_a), int(trans_b), _ptr(a), _ptr(b), _ptr(c), _dtype_code(a),
                                      _dtype_code(c), alpha, beta, _ptr(workspace), ws_bytes, _stream(stream)))


def oomb_bias_rope(x_in, bias, x_out, n_heads: int, pos0: int, theta: float, mode: int, stream=None) -> None:
    """x_out[i, h, :] = rotation(pos0 + i) (x_in[i, h, :] + bias[h, :]); mode 0 none, 1 forward, 2 inverse."""
    n = x_in.shape[0]
    d = x_in.numel() // (n * n_heads)
    _ok("oomb_bias_rope", load().oomb_bias_rope(_ptr(x_in), _dtype_code(x_in), _ptr(bias), _ptr(x_out),
                                                _dtype_code(x_out), n, n_heads, d, pos0, theta, mode,
                                                _stream(stream)))


def oomb_bias_rope_axes(x_in, bias, x_out, n_heads: int, positions, pair_axis, theta: float, mode: int,
                        own_ladder: bool = False, stream=None) -> None:
    """oomb_bias_rope with positions [n_axes, n] (int64); pair_axis[j] is the axis of pair j (d/2 entries)."""
    import torch
    f, dev = "oomb_bias_rope_axes", torch.cuda.current_device()
    ti, to = _dtype_code(x_in), _dtype_code(x_out)
    total, n = x_in.numel(), x_in.shape[0] if x_in.dim() else 0
    if n <= 0 or n_heads <= 0 or total == 0 or total % (n * n_heads) or x_out.numel() != total:
        raise ValueError(f"{f}: x_in {tuple(x_in.shape)} and x_out {tuple(x_out.shape)} do not hold rows of "
                         f"{n_heads} heads")
    d = total // (n * n_heads)
    a_in, a_out = _need(f, "x_in", x_in, x_in.shape, x_in.dtype, dev), _need(f, "x_out", x_out, x_out.shape, x_out.dtype, dev)
    if bias is not None and bias.numel() != n_heads * d:
        raise ValueError(f"{f}: bias has {bias.numel()} elements, needs {n_heads * d}")
    a_bias = None if bias is None else _need(f, "bias", bias, bias.shape, torch.float32, dev)
    axes, a_pos, n_axes = None, None, 0
    if mode != 0:
        axes = pair_axis if isinstance(pair_axis, bytes) else bytes(list(pair_axis))
        if 2 * len(axes) != d:
            raise ValueError(f"{f}: pair_axis has {len(axes)} entries, needs {d // 2}")
        n_axes = _dims(f, "positions", positions, 2)[0]
        a_pos = _need(f, "positions", positions, (n_axes, n), torch.int64, dev)
    _ok(f, load().oomb_bias_rope_axes(a_in, ti, a_bias, a_out, to, n, n_heads, d, a_pos, n_axes, axes, theta,
                                      int(own_ladder), mode, _stream(stream)))


def _norm_call(f: str, x, y, w_pre, w_post, gate, dev: int):
    """Checks the inputs common to both directions; (n, D, gate_rows, addresses)."""
    import torch
    f32, dt = torch.float32, x.dtype
    n, D = shape = _dims(f, "x", x, 2)
    rows = gate is not None and gate.dim() == 2
    return n, D, int(rows), (_need(f, "x", x, shape, dt, dev), _opt(f, "y", y, shape, dt, dev),
                             _opt(f, "w_post", w_post, (D,), f32, dev),
                             _opt(f, "gate", gate, shape if rows else (D,), dt if rows else f32, dev),
                             _opt(f, "w_pre", w_pre, (D,), f32, dev))


def oomb_block_norm_fwd(x, y, x_out, u=None, w_pre=None, w_post=None, gate=None, res_scale: float = 1.0,
                        eps: float = 1e-6, rstd_pre=None, rstd_post=None, stream=None) -> None:
    """x_out = x + res_scale * gate * norm(y; w_post), u = norm(x_out; w_pre).  gate: fp32 [D] or [n, D] like x."""
    import torch
    f, dev, f32, dt = "oomb_block_norm_fwd", torch.cuda.current_device(), torch.float32, x.dtype
    n, D, rows, (ax, ay, awp, ag, aw) = _norm_call(f, x, y, w_pre, w_post, gate, dev)
    _ok(f, load().oomb_block_norm_fwd(ax, ay, awp, ag, rows, aw, res_scale, eps, n, D, _dtype_code(x),
                                      _opt(f, "x_out", x_out, (n, D), dt, dev), _opt(f, "u", u, (n, D), dt, dev),
                                      _opt(f, "rstd_post", rstd_post, (n,), f32, dev),
                                      _opt(f, "rstd_pre", rstd_pre, (n,), f32, dev), _stream(stream)))


def oomb_block_norm_bwd(x, y, dx, dy=None, du=None, dx_out=None, rstd_pre=None, rstd_post=None, w_pre=None,
                        w_post=None, gate=None, dw_pre=None, dw_post=None, dgate=None, res_scale: float = 1.0,
                        accumulate: bool = False, workspace=None, stream=None) -> None:
    """The backward of oomb_block_norm_fwd; accumulate adds the parameter gradients to their buffers."""
    import torch
    f, dev, f32, dt = "oomb_block_norm_bwd", torch.cuda.current_device(), torch.float32, x.dtype
    n, D, rows, (ax, ay, awp, ag, aw) = _norm_call(f, x, y, w_pre, w_post, gate, dev)
    shape = (n, D)
    ws, ws_bytes = _scratch(f, workspace, dev)
    _ok(f, load().oomb_block_norm_bwd(ax, ay, awp, ag, rows, aw, res_scale, n, D, _dtype_code(x),
                                      _opt(f, "rstd_post", rstd_post, (n,), f32, dev),
                                      _opt(f, "rstd_pre", rstd_pre, (n,), f32, dev), _opt(f, "du", du, shape, dt, dev),
                                      _opt(f, "dx_out", dx_out, shape, dt, dev), _need(f, "dx", dx, shape, dt, dev),
                                      _opt(f, "dy", dy, shape, dt, dev), _opt(f, "dw_post", dw_post, (D,), f32, dev),
                                      _opt(f, "dgate", dgate, shape if rows else (D,), dt if rows else f32, dev),
                                      _opt(f, "dw_pre", dw_pre, (D,), f32, dev), int(accumulate), ws, ws_bytes,
                                      _stream(stream)))


def oomb_block_norm_workspace(n: int, D: int) -> int:
    return int(load().oomb_block_norm_workspace(n, D))


def oomb_block_norm_check(stream=None) -> int:
    """Raises OombError if a block norm of the current device gave up waiting since the last check."""
    bits = C.c_uint32(0)
    _ok("oomb_block_norm_check", load().oomb_block_norm_check(_stream(stream), C.byref(bits)))
    return bits.value


def oomb_block_norm_test_timeout(on: bool) -> None:
    """For tests: while on, the first row of calls with many rows never comes, and they give up on it."""
    load().oomb_block_norm_test_timeout(int(on))


def _word(func: str, t, dev: int) -> int:
    """Address of a caller's device error word: the first of one or more 32-bit integers."""
    import torch
    if t is None:
        raise ValueError(f"{func}: error_word is missing")
    if t.dtype is not torch.int32 and t.dtype is not torch.uint32:
        raise TypeError(f"{func}: error_word has to be 32-bit integers, not {t.dtype}")
    if t.numel() < 1:
        raise ValueError(f"{func}: error_word is empty")
    if t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _need(func, "error_word", t, t.shape, t.dtype, dev)


def _lead(func: str, name: str, t, n: int, dev: int):
    """Shape and address of a tensor that sets the sizes the others are checked against."""
    if t is None or len(shape := t.shape) != n:
        raise ValueError(f"{func}: {name} has to have {n} dimensions")
    if t.get_device() == dev and t.is_contiguous():
        return shape, t.data_ptr()
    return shape, _need(func, name, t, shape, t.dtype, dev)


def _code(torch, t) -> int:
    return OOMB_BF16 if t.dtype is torch.bfloat16 else OOMB_FP32 if t.dtype is torch.float32 else _dtype_code(t)


def _on(torch, stream, dev: int):
    """Raw stream of a call on device ``dev``."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) if stream is None else None
    return _stream(stream) if raw is None else raw(dev)


def oomb_embed_fwd(tokens, table, out, error_word, scale: float = 1.0, stream=None) -> None:
    """out[i] = scale * table[tokens[i]] (int64 tokens; a negative one is none: a row of zeros)."""
    import torch
    f, dev = "oomb_embed_fwd", torch.cuda.current_device()
    n = _dims(f, "tokens", tokens, 1)[0]
    code = _code(torch, table)
    at = _need(f, "tokens", tokens, (n,), torch.int64, dev)
    (V, D), atab = _lead(f, "table", table, 2, dev)
    _ok(f, load().oomb_embed_fwd(at, n, atab, V, D, code, scale, _need(f, "out", out, (n, D), table.dtype, dev),
                                 _word(f, error_word, dev), _on(torch, stream, dev)))


def oomb_embed_bwd(tokens, d_out, d_table, workspace, error_word, scale: float = 1.0, accumulate: bool = False,
                   stream=None) -> None:
    """d_table[t] (fp32) = (accumulate: +=) scale * the sum of d_out over the rows of token t."""
    import torch
    f, dev = "oomb_embed_bwd", torch.cuda.current_device()
    n = _dims(f, "tokens", tokens, 1)[0]
    V, D = _dims(f, "d_table", d_table, 2)
    ws, ws_bytes = _scratch(f, workspace, dev)
    _ok(f, load().oomb_embed_bwd(_need(f, "tokens", tokens, (n,), torch.int64, dev), n,
                                 _need(f, "d_out", d_out, (n, D), d_out.dtype, dev), V, D, _code(torch, d_out), scale,
                                 _need(f, "d_table", d_table, (V, D), torch.float32, dev), int(accumulate), ws, ws_bytes,
                                 _word(f, error_word, dev), _on(torch, stream, dev)))


def oomb_embed_workspace(n: int, D: int) -> int:
    return int(load().oomb_embed_workspace(n, D))


def oomb_layer_norm_fwd(x, w, b, out, eps: float = 1e-5, mean=None, rstd=None, stream=None) -> None:
    """out = (x - mean) * rstd * w + b over the rows of x [n, D]; w and b fp32 [D] or None."""
    import torch
    f, dev, f32 = "oomb_layer_norm_fwd", torch.cuda.current_device(), torch.float32
    shape, ax = _lead(f, "x", x, 2, dev)
    n, D = shape
    _ok(f, load().oomb_layer_norm_fwd(ax, _opt(f, "w", w, (D,), f32, dev), _opt(f, "b", b, (D,), f32, dev), eps, n, D,
                                      _code(torch, x), _need(f, "out", out, shape, x.dtype, dev),
                                      _opt(f, "mean", mean, (n,), f32, dev), _opt(f, "rstd", rstd, (n,), f32, dev),
                                      _on(torch, stream, dev)))


def oomb_layer_norm_bwd(x, w, mean, rstd, dy, dx, dw=None, db=None, dx_out=None, accumulate: bool = False,
                        workspace=None, stream=None) -> None:
    """The backward of oomb_layer_norm_fwd; accumulate adds the parameter gradients to their buffers.  Without dw and
    db no workspace is needed."""
    import torch
    f, dev, f32 = "oomb_layer_norm_bwd", torch.cuda.current_device(), torch.float32
    shape, ax = _lead(f, "x", x, 2, dev)
    n, D = shape
    dt = x.dtype
    ws, ws_bytes = _scratch(f, workspace, dev)
    _ok(f, load().oomb_layer_norm_bwd(ax, _opt(f, "w", w, (D,), f32, dev), _need(f, "mean", mean, (n,), f32, dev),
                                      _need(f, "rstd", rstd, (n,), f32, dev), _need(f, "dy", dy, shape, dt, dev),
                                      _opt(f, "dx_out", dx_out, shape, dt, dev), n, D, _code(torch, x),
                                      _need(f, "dx", dx, shape, dt, dev), _opt(f, "dw", dw, (D,), f32, dev),
                                      _opt(f, "db", db, (D,), f32, dev), int(accumulate), ws, ws_bytes,
                                      _on(torch, stream, dev)))


def oomb_layer_norm_workspace(n: int, D: int) -> int:
    return int(load().oomb_layer_norm_workspace(n, D))


def _head_call(torch, f: str, x, w, targets, dev: int):
    """Checks the inputs common to both directions; (n, D, V, dtype code, addresses)."""
    n, D = _dims(f, "x", x, 2)
    V = _dims(f, "w", w, 2)[0]
    code = _code(torch, x)
    ax = _lead(f, "x", x, 2, dev)[1]
    return n, D, V, code, (ax, _need(f, "w", w, (V, D), x.dtype, dev), _need(f, "targets", targets, (n,), torch.int64, dev))


def oomb_head_loss_fwd(x, w, targets, loss, lse, workspace, error_word, softcap: float = 0.0, stream=None) -> None:
    """loss[i] = lse[i] - z[i, targets[i]] of the logits z = x w^T, which are not kept (targets int64 [n];
    a negative one is none: loss and lse are 0)."""
    import torch
    f, dev, f32 = "oomb_head_loss_fwd", torch.cuda.current_device(), torch.float32
    n, D, V, code, (ax, aw, at) = _head_call(torch, f, x, w, targets, dev)
    ws, ws_bytes = _scratch(f, workspace, dev)
    _ok(f, load().oomb_head_loss_fwd(ax, aw, at, n, D, V, code, softcap, _need(f, "loss", loss, (n,), f32, dev),
                                     _need(f, "lse", lse, (n,), f32, dev), ws, ws_bytes, _word(f, error_word, dev),
                                     _on(torch, stream, dev)))


def oomb_head_loss_bwd(x, w, targets, lse, dx, dw, workspace, error_word, d_loss=None, scale: float = 1.0,
                       softcap: float = 0.0, accumulate: bool = False, stream=None) -> None:
    """dx (like x, or None) and dw (like w or fp32, or None; accumulate adds to an fp32 one) for the
    gradient scale * d_loss[i] of loss[i] (d_loss fp32 [n]; None: 1)."""
    import torch
    f, dev, f32 = "oomb_head_loss_bwd", torch.cuda.current_device(), torch.float32
    n, D, V, code, (ax, aw, at) = _head_call(torch, f, x, w, targets, dev)
    ws, ws_bytes = _scratch(f, workspace, dev)
    dw_code = code if dw is None else _code(torch, dw)
    _ok(f, load().oomb_head_loss_bwd(ax, aw, at, _need(f, "lse", lse, (n,), f32, dev),
                                     _opt(f, "d_loss", d_loss, (n,), f32, dev), scale, n, D, V, code, softcap,
                                     _opt(f, "dx", dx, (n, D), x.dtype, dev),
                                     None if dw is None else _need(f, "dw", dw, (V, D), dw.dtype, dev), dw_code,
                                     int(accumulate), ws, ws_bytes, _word(f, error_word, dev), _on(torch, stream, dev)))


def oomb_head_loss_workspace(n: int, D: int, V: int, dtype, backward: bool) -> int:
    """Bytes for calls of up to n rows; dtype: the tensors' (torch.bfloat16 or torch.float32), or its code."""
    import torch
    code = {torch.bfloat16: OOMB_BF16, torch.float32: OOMB_FP32}.get(dtype, dtype)
    if not isinstance(code, int):
        raise TypeError(f"unsupported dtype {dtype}")
    return int(load().oomb_head_loss_workspace(n, D, V, code, int(backward)))


def oomb_word_check(error_word, stream=None) -> int:
    """Raises OombError if kernels have set bits in this device error word since the last check; clears it."""
    import torch
    bits = C.c_uint32(0)
    st = load().oomb_word_check(_word("oomb_word_check", error_word, torch.cuda.current_device()), _stream(stream),
                                C.byref(bits))
    if st == 7:
        _ok("oomb_word_check", st)
    if st != 0:
        raise OombError("oomb_word_check", st, f"device error bits 0x{bits.value:x}")
    return bits.value


def oomb_grad_gather(pool: int, first_token: int, dk, dv, stream=None) -> None:
    _ok("oomb_grad_gather", load().oomb_grad_gather(pool, first_token, dk.shape[0], _ptr(dk), _ptr(dv),
                                                    _stream(stream)))


def oomb_grad_prefetch(pool: int, sel, sel_count, prev_sel, prev_count, stage_buf: int, stream=None) -> None:
    _ok("oomb_grad_prefetch", load().oomb_grad_prefetch(pool, _ptr(sel), _ptr(sel_count), sel.shape[-1],
                                                        _ptr(prev_sel), _ptr(prev_count), stage_buf,
                                                        _stream(stream)))


def oomb_grad_carry(pool: int, sel, sel_count, prev_sel, prev_count, stage_buf: int, stream=None) -> None:
    _ok("oomb_grad_carry", load().oomb_grad_carry(pool, _ptr(sel), _ptr(sel_count), sel.shape[-1], _ptr(prev_sel),
                                                  _ptr(prev_count), stage_buf, _stream(stream)))


def oomb_grad_writeback(pool: int, sel, sel_count, stage_buf: int, stream=None) -> None:
    _ok("oomb_grad_writeback", load().oomb_grad_writeback(pool, _ptr(sel), _ptr(sel_count), sel.shape[-1],
                                                          stage_buf, _stream(stream)))


def oomb_prefetch_pages(pool: int, sel, sel_count, stage_buf: int, first_page: int, end_page: int,
                        stream=None) -> None:
    _ok("oomb_prefetch_pages", load().oomb_prefetch_pages(pool, _ptr(sel), _ptr(sel_count), sel.shape[-1], stage_buf,
                                                          first_page, end_page, _stream(stream)))


def oomb_pool_set_stage(pool: int, stage_buf: int) -> None:
    _ok("oomb_pool_set_stage", load().oomb_pool_set_stage(pool, stage_buf))


def oomb_workspace_size(pool: int, op: int, n_q: int) -> int:
    return int(load().oomb_workspace_size(pool, op, n_q))


def oomb_check(pool: int, stream=None) -> int:
    bits = C.c_uint32(0)
    st = load().oomb_check(pool, _stream(stream), C.byref(bits))
    if st != 0:
        raise OombError("oomb_check", st, f"device error bits 0x{bits.value:x}")
    return bits.value


def oomb_page_table_host(pool: int, n: int):
    buf = (C.c_int32 * n)()
    m = load().oomb_page_table_host(pool, buf, n)
    return list(buf)[:m]


def oomb_pool_tokens(pool: int) -> int:
    return int(load().oomb_pool_tokens(pool))


def oomb_pool_free_pages(pool: int) -> int:
    return int(load().oomb_pool_free_pages(pool))


def oomb_uses_tensor_cores(pool: int) -> bool:
    return bool(load().oomb_uses_tensor_cores(pool))


def oomb_launch_count() -> int:
    return int(load().oomb_launch_count())


OOMB_APPEND_POOL, OOMB_APPEND_STAGED, OOMB_APPEND_DEFERRED = 0, 1, 2


def oomb_page_select_append(pool: int, q, k, v, q_start: int, top_k: int, n_sink: int, sel, sel_count, workspace,
                            append_mode: int = OOMB_APPEND_POOL, stage_buf: int = 0, n_q: Optional[int] = None,
                            stream=None) -> None:
    """oomb_page_select and the append of the chunk's K/V (the chunk's tokens) in one call."""
    n = q.shape[0] if n_q is None else n_q
    ws_bytes = workspace.numel() * workspace.element_size()
    _ok("oomb_page_select_append", load().oomb_page_select_append(pool, _ptr(q), _ptr(k), _ptr(v), q_start, n, top_k,
                                                                  n_sink, _ptr(sel), _ptr(sel_count), sel.shape[-1],
                                                                  _ptr(workspace), ws_bytes, append_mode, stage_buf,
                                                                  _stream(stream)))


def oomb_page_select_noalloc(pool: int, q, q_start: int, top_k: int, n_sink: int, sel, sel_count,
                             n_q: Optional[int] = None, stream=None) -> None:
    """oomb_page_select with the library's static scratch instead of a workspace."""
    n = q.shape[0] if n_q is None else n_q
    _ok("oomb_page_select_noalloc", load().oomb_page_select_noalloc(pool, _ptr(q), q_start, n, top_k, n_sink,
                                                                    _ptr(sel), _ptr(sel_count), sel.shape[-1],
                                                                    _stream(stream)))
