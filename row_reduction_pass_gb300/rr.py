"""Thin ctypes binding of ``librr.so`` (the C ABI declared in ``include/rr.h``).

Argument marshalling only: every function takes torch tensors (device memory),
passes their pointers, sizes, the dtype code and the current CUDA stream to the
C entry point of the same name, and raises :class:`RRError` on a non-zero
status.  No arithmetic of the method happens here, and there is no fallback:
if the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIBNAME = "librr.so"
_lock = threading.Lock()
_lib = None
_torch_module = None  # imported at the first call

RR_F32 = 0
RR_BF16 = 1

_STATUS = {
    0: "RR_OK", 1: "RR_ERR_INVALID_ARG", 2: "RR_ERR_UNSUPPORTED_DTYPE",
    3: "RR_ERR_ALIASING", 4: "RR_ERR_WORKSPACE_TOO_SMALL", 5: "RR_ERR_CUDA",
    6: "RR_ERR_DEVICE_TIMEOUT",
}


class RRError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)} ({msg})")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, _LIBNAME)


def load_library():
    """Load librr.so (built by ``__graft_entry__.build()``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        st = ctypes.c_int
        lib.rr_status_string.argtypes = [st]
        lib.rr_status_string.restype = ctypes.c_char_p
        lib.rr_softmax_fwd.argtypes = [vp, vp, i64, i64, st, vp]
        lib.rr_softmax_fwd.restype = st
        lib.rr_softmax_xent_fwd_bwd.argtypes = [vp, vp, vp, vp, i64, i64, i32, vp, st, vp]
        lib.rr_softmax_xent_fwd_bwd.restype = st
        lib.rr_log_softmax_fwd.argtypes = [vp, vp, i64, i64, st, vp]
        lib.rr_log_softmax_fwd.restype = st
        lib.rr_softmax_bwd.argtypes = [vp, vp, vp, i64, i64, st, vp]
        lib.rr_softmax_bwd.restype = st
        lib.rr_log_softmax_bwd.argtypes = [vp, vp, vp, i64, i64, st, vp]
        lib.rr_log_softmax_bwd.restype = st
        lib.rr_layernorm_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, ctypes.c_float,
                                         st, vp]
        lib.rr_layernorm_fwd.restype = st
        lib.rr_layernorm_bwd_workspace_size.argtypes = [i64, i64, st]
        lib.rr_layernorm_bwd_workspace_size.restype = ctypes.c_size_t
        lib.rr_layernorm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                         i64, i64, st, vp]
        lib.rr_layernorm_bwd.restype = st
        lib.rr_rmsnorm_fwd.argtypes = [vp, vp, vp, vp, i64, i64, ctypes.c_float, st, vp]
        lib.rr_rmsnorm_fwd.restype = st
        lib.rr_rmsnorm_bwd_workspace_size.argtypes = [i64, i64, st]
        lib.rr_rmsnorm_bwd_workspace_size.restype = ctypes.c_size_t
        lib.rr_rmsnorm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, i64, i64, st,
                                       vp]
        lib.rr_rmsnorm_bwd.restype = st
        lib.rr_layernorm_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, st, vp]
        lib.rr_layernorm_bwd_noalloc.restype = st
        lib.rr_last_error_detail.argtypes = []
        lib.rr_last_error_detail.restype = ctypes.c_char_p
        lib.rr_read_device_error.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int), st]
        lib.rr_read_device_error.restype = st
        lib.rr_selftest_bounded_wait.argtypes = [i64, vp]
        lib.rr_selftest_bounded_wait.restype = st
        lib.rr_attention_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_float,
                                         ctypes.c_int, st, vp]
        lib.rr_attention_fwd.restype = st
        f32 = ctypes.c_float
        lib.rr_distill_fwd_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, f32,
                                           ctypes.c_int, vp, st, vp]
        lib.rr_distill_fwd_bwd.restype = st
        lib.rr_attention_tree_workspace_size.argtypes = [i64, i64, i64, i64, i64]
        lib.rr_attention_tree_workspace_size.restype = ctypes.c_size_t
        lib.rr_attention_tree_fwd.argtypes = [vp] * 9 + [ctypes.c_size_t] + [i64] * 8 + [f32, st,
                                                                                        vp]
        lib.rr_attention_tree_fwd.restype = st
        lib.rr_draft_verify.argtypes = [vp] * 10 + [i64, i64, i64, st, vp]
        lib.rr_draft_verify.restype = st
        _lib = lib
        return lib


def rr_status_string(status: int) -> str:
    return load_library().rr_status_string(int(status)).decode()


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _check(fn: str, status: int):
    if status != 0:
        detail = load_library().rr_last_error_detail()
        raise RRError(fn, status, (detail or b"").decode())


def _dtype(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return RR_F32
    if t.dtype == torch.bfloat16:
        return RR_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(stream):
    """The stream's handle; the current one's without building a Stream object
    (3 us of a call's 12-17)."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous row-major")


def rr_softmax_fwd(x, y, stream=None):
    """y[r, :] = softmax(x[r, :]); y may be x (in place)."""
    _contig(x, y)
    rows, cols = x.shape
    _check("rr_softmax_fwd", load_library().rr_softmax_fwd(
        _p(x), _p(y), rows, cols, _dtype(x), _stream(stream)))


def rr_softmax_xent_fwd_bwd(logits, labels, loss, dlogits, ignore_index=-100,
                            bad_label_count=None, stream=None):
    """Per-row loss (fp32) and dlogits = softmax - onehot; dlogits may be logits."""
    _contig(logits, labels, loss, dlogits)
    rows, cols = logits.shape
    _check("rr_softmax_xent_fwd_bwd", load_library().rr_softmax_xent_fwd_bwd(
        _p(logits), _p(labels), _p(loss), _p(dlogits), rows, cols, int(ignore_index),
        _p(bad_label_count), _dtype(logits), _stream(stream)))


def rr_log_softmax_fwd(x, z, stream=None):
    """z = log_softmax(x) per row (z may be x)."""
    _contig(x, z)
    rows, cols = x.shape
    _check("rr_log_softmax_fwd", load_library().rr_log_softmax_fwd(
        _p(x), _p(z), rows, cols, _dtype(x), _stream(stream)))


def rr_softmax_bwd(y, dy, dx, stream=None):
    """dx = y * (dy - sum(y * dy)) per row, y the softmax output."""
    _contig(y, dy, dx)
    rows, cols = y.shape
    _check("rr_softmax_bwd", load_library().rr_softmax_bwd(
        _p(y), _p(dy), _p(dx), rows, cols, _dtype(y), _stream(stream)))


def rr_log_softmax_bwd(z, dz, dx, stream=None):
    """dx = dz - exp(z) * sum(dz) per row, z the log-softmax output."""
    _contig(z, dz, dx)
    rows, cols = z.shape
    _check("rr_log_softmax_bwd", load_library().rr_log_softmax_bwd(
        _p(z), _p(dz), _p(dx), rows, cols, _dtype(z), _stream(stream)))


def rr_attention_fwd(q, k, v, o, lse=None, scale=None, causal=True, stream=None):
    """Scaled dot-product attention of [bh, seq, head_dim] bf16 tensors:
    o = softmax(scale * q k^T (causal mask)) v, lse (fp32 [bh, seq]) optional;
    scale defaults to 1 / sqrt(head_dim)."""
    _contig(q, k, v, o)
    if lse is not None:
        _contig(lse)
    bh, seq, d = q.shape
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    _check("rr_attention_fwd", load_library().rr_attention_fwd(
        _p(q), _p(k), _p(v), _p(o), _p(lse), bh, seq, d, ctypes.c_float(scale),
        1 if causal else 0, _dtype(q), _stream(stream)))


def rr_layernorm_fwd(x, gamma, beta, y, mean, rstd, eps=1e-5, stream=None):
    """y = (x - mean) * rstd * gamma + beta; saves mean and rstd (fp32)."""
    _contig(x, gamma, beta, y, mean, rstd)
    rows, cols = x.shape
    _check("rr_layernorm_fwd", load_library().rr_layernorm_fwd(
        _p(x), _p(gamma), _p(beta), _p(y), _p(mean), _p(rstd), rows, cols,
        ctypes.c_float(eps), _dtype(x), _stream(stream)))


def rr_layernorm_bwd_workspace_size(rows: int, cols: int, dtype) -> int:
    import torch
    code = {torch.float32: RR_F32, torch.bfloat16: RR_BF16}.get(dtype, dtype)
    return int(load_library().rr_layernorm_bwd_workspace_size(rows, cols, int(code)))


def rr_layernorm_bwd(dy, x, mean, rstd, gamma, dx, dgamma, dbeta, workspace=None,
                     stream=None):
    """dx, dgamma, dbeta of LayerNorm from the saved mean / rstd.

    ``workspace`` is a uint8 CUDA tensor of at least
    ``rr_layernorm_bwd_workspace_size`` bytes; it is allocated here if omitted."""
    import torch
    _contig(dy, x, mean, rstd, gamma, dx, dgamma, dbeta)
    rows, cols = x.shape
    need = rr_layernorm_bwd_workspace_size(rows, cols, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check("rr_layernorm_bwd", load_library().rr_layernorm_bwd(
        _p(dy), _p(x), _p(mean), _p(rstd), _p(gamma), _p(dx), _p(dgamma), _p(dbeta),
        _p(workspace), workspace.numel() * workspace.element_size(), rows, cols,
        _dtype(x), _stream(stream)))


def rr_layernorm_bwd_noalloc(dy, x, mean, rstd, gamma, dx, dgamma, dbeta, stream=None):
    """rr_layernorm_bwd without a workspace argument: the library's fixed 8 MiB
    scratch holds the column partials (for callers that cannot allocate).
    Calls on one device must not overlap on the GPU."""
    _contig(dy, x, mean, rstd, gamma, dx, dgamma, dbeta)
    rows, cols = x.shape
    _check("rr_layernorm_bwd_noalloc", load_library().rr_layernorm_bwd_noalloc(
        _p(dy), _p(x), _p(mean), _p(rstd), _p(gamma), _p(dx), _p(dgamma), _p(dbeta), rows, cols,
        _dtype(x), _stream(stream)))


def rr_rmsnorm_fwd(x, gamma, y, rstd, eps=1e-5, stream=None):
    """y = x * rstd * gamma with rstd = 1/sqrt(mean(x^2) + eps) (fp32, saved)."""
    _contig(x, gamma, y, rstd)
    rows, cols = x.shape
    _check("rr_rmsnorm_fwd", load_library().rr_rmsnorm_fwd(
        _p(x), _p(gamma), _p(y), _p(rstd), rows, cols, ctypes.c_float(eps), _dtype(x),
        _stream(stream)))


def rr_rmsnorm_bwd_workspace_size(rows: int, cols: int, dtype) -> int:
    import torch
    code = {torch.float32: RR_F32, torch.bfloat16: RR_BF16}.get(dtype, dtype)
    return int(load_library().rr_rmsnorm_bwd_workspace_size(rows, cols, int(code)))


def rr_rmsnorm_bwd(dy, x, rstd, gamma, dx, dgamma, workspace=None, stream=None):
    """dx and dgamma of RMSNorm from the saved rstd.

    ``workspace`` is a uint8 CUDA tensor of at least
    ``rr_rmsnorm_bwd_workspace_size`` bytes; it is allocated here if omitted."""
    import torch
    _contig(dy, x, rstd, gamma, dx, dgamma)
    rows, cols = x.shape
    need = rr_rmsnorm_bwd_workspace_size(rows, cols, x.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check("rr_rmsnorm_bwd", load_library().rr_rmsnorm_bwd(
        _p(dy), _p(x), _p(rstd), _p(gamma), _p(dx), _p(dgamma), _p(workspace),
        workspace.numel() * workspace.element_size(), rows, cols, _dtype(x), _stream(stream)))


def _args(fn, *ts):
    """Checks (name, tensor, dtype or None, shape) tuples of one call: contiguous
    CUDA tensors of that dtype and shape on the current device (a None tensor,
    an absent argument, passes).  Returns their addresses."""
    out, devs = [], set()
    for name, t, dtype, shape in ts:
        if t is None:
            out.append(None)
            continue
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"{fn}: {name} must be {dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{fn}: {name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous")
        out.append(t.data_ptr())
        devs.add(t.get_device())
    if len(devs) != 1 or -1 in devs or devs != {_torch().cuda.current_device()}:
        for name, t, _, _ in ts:
            if t is not None and not t.is_cuda:
                raise ValueError(f"{fn}: {name} must be a CUDA tensor")
        raise ValueError(f"{fn}: the tensors must all be on the current device")
    return out


def rr_distill_fwd_bwd(logits, top_index, top_value, loss, dlogits=None, grad=None,
                       temperature=1.0, tail=False, bad_index_count=None, stream=None):
    """Distillation loss (fp32 [rows]) and dlogits from a teacher's top entries
    (top_index int32, top_value fp32, [rows, k]); tail keeps the teacher's mass
    outside the list (top_value then holds log-probabilities).  dlogits may be
    logits, or None for the loss alone; grad [rows] scales dlogits."""
    torch = _torch()
    rows, cols = logits.shape
    k = top_index.shape[1]
    i32, f32 = torch.int32, torch.float32
    fn = "rr_distill_fwd_bwd"
    if bad_index_count is not None and bad_index_count.numel() != 1:
        raise ValueError(f"{fn}: bad_index_count must hold one value")
    x, i, v, l, d, g, bad = _args(
        fn, ("logits", logits, None, (rows, cols)), ("top_index", top_index, i32, (rows, k)),
        ("top_value", top_value, f32, (rows, k)), ("loss", loss, f32, (rows,)),
        ("dlogits", dlogits, logits.dtype, (rows, cols)), ("grad", grad, f32, (rows,)),
        ("bad_index_count", bad_index_count, i32,
         None if bad_index_count is None else bad_index_count.shape))
    st = load_library().rr_distill_fwd_bwd(x, i, v, g, l, d, rows, cols, k, temperature,
                                           1 if tail else 0, bad, _dtype(logits),
                                           _raw_stream(stream))
    if st != 0:
        _check(fn, st)


def rr_attention_tree_workspace_size(batch: int, nodes: int, heads: int, kv_heads: int,
                                     head_dim: int) -> int:
    return int(load_library().rr_attention_tree_workspace_size(batch, nodes, heads, kv_heads,
                                                               head_dim))


def rr_attention_tree_fwd(q, k_cache, v_cache, page_table, context_len, o, lse=None, parents=None,
                          scale=None, workspace=None, stream=None):
    """Attention of the new tokens q [batch, nodes, heads, head_dim] (bf16) over
    a paged cache [pages, page_size, kv_heads, head_dim] that already holds their
    keys and values: node j of sequence b at position context_len[b] + j, position
    p on page page_table[b, p // page_size].  parents [batch, nodes] makes them a
    tree (None: a chain, node i sees the nodes up to i); lse (fp32) is optional;
    scale defaults to 1 / sqrt(head_dim).

    ``workspace`` is a uint8 CUDA tensor of at least
    ``rr_attention_tree_workspace_size`` bytes; it is allocated here if omitted."""
    torch = _torch()
    b, n, h, d = q.shape
    pages, page_size, kv, _ = k_cache.shape
    width = page_table.shape[1]
    i32, dt, cache = torch.int32, q.dtype, (pages, page_size, kv, d)
    fn = "rr_attention_tree_fwd"
    lib = load_library()
    pq, pk, pv, pt, pc, po, pl, pp, pw = _args(
        fn, ("q", q, None, (b, n, h, d)), ("k_cache", k_cache, dt, cache),
        ("v_cache", v_cache, dt, cache), ("page_table", page_table, i32, (b, width)),
        ("context_len", context_len, i32, (b,)), ("o", o, dt, (b, n, h, d)),
        ("lse", lse, torch.float32, (b, n, h)), ("parents", parents, i32, (b, n)),
        ("workspace", workspace, None, None if workspace is None else workspace.shape))
    if workspace is None:
        need = lib.rr_attention_tree_workspace_size(b, n, h, kv, d)
        if need > 0:
            if stream is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            else:  # of the stream that uses it
                with torch.cuda.stream(stream):
                    workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            pw = workspace.data_ptr()
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if scale is None:
        scale = 1.0 / float(d) ** 0.5
    st = lib.rr_attention_tree_fwd(pq, pk, pv, pt, pc, pp, po, pl, pw, size, b, n, h, kv, d, pages,
                                   page_size, width, scale, _dtype(q), _raw_stream(stream))
    if st != 0:
        _check(fn, st)


def rr_draft_verify(target_logits, draft_logits, tokens, uniform, race, out_tokens, out_nodes,
                    out_count, parents=None, temperature=None, stream=None):
    """Accepts drafted tokens against the target's probabilities, along the
    chain or tree they form, and draws the token that follows them.

    target_logits [batch, nodes + 1, cols], draft_logits [batch, nodes, cols],
    tokens / parents (int32) and uniform (fp32) [batch, nodes], race [batch, cols]
    exponential noise, temperature [batch] (<= 0: greedy, each distribution all on its
    largest logit).  Writes out_tokens and
    out_nodes [batch, nodes + 1] and out_count [batch] (int32)."""
    torch = _torch()
    b, n1, v = target_logits.shape
    n, dt, i32, f32 = n1 - 1, target_logits.dtype, torch.int32, torch.float32
    fn = "rr_draft_verify"
    pt, pd, pk, pp, pu, pr, pT, ot, on, oc = _args(
        fn, ("target_logits", target_logits, None, (b, n1, v)),
        ("draft_logits", draft_logits, dt, (b, n, v)), ("tokens", tokens, i32, (b, n)),
        ("parents", parents, i32, (b, n)), ("uniform", uniform, f32, (b, n)),
        ("race", race, f32, (b, v)), ("temperature", temperature, f32, (b,)),
        ("out_tokens", out_tokens, i32, (b, n1)), ("out_nodes", out_nodes, i32, (b, n1)),
        ("out_count", out_count, i32, (b,)))
    st = load_library().rr_draft_verify(pt, pd, pk, pp, pu, pr, pT, ot, on, oc, b, n, v,
                                        _dtype(target_logits), _raw_stream(stream))
    if st != 0:
        _check(fn, st)


def rr_read_device_error(device: int = 0, reset: bool = True) -> int:
    """Device-side error word (0 = none, else an RR status such as a timed-out wait)."""
    out = ctypes.c_int(0)
    _check("rr_read_device_error", load_library().rr_read_device_error(
        int(device), ctypes.byref(out), int(bool(reset))))
    return out.value


def rr_selftest_bounded_wait(limit_ns: int, stream=None):
    """Launch the bounded-wait self-test: one block waits on an mbarrier that
    nothing completes, gives up after ``limit_ns`` and records
    RR_ERR_DEVICE_TIMEOUT in the device error word (read it with
    :func:`rr_read_device_error`)."""
    _check("rr_selftest_bounded_wait", load_library().rr_selftest_bounded_wait(
        int(limit_ns), _stream(stream)))
