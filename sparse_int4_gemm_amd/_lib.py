"""ctypes binding of libslim.so (include/slim.h).

Argument marshalling only: every function passes device pointers, sizes and
the current HIP stream to the C ABI; all computation runs in the library's
HIP kernels.  PyTorch supplies device memory and streams.  There is no
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("SLIM_LIB", os.path.join(_HERE, "libslim.so"))

SLIM_OK = 0
SLIM_EINVAL = 1
SLIM_EUNSUPPORTED = 2
SLIM_EHIP = 3

EXPORTED = (
    "slim_status_string", "slim_last_error", "slim_version",
    "slim_values_bytes", "slim_meta_bytes", "slim_scales_bytes",
    "slim_pack", "slim_linear_workspace_bytes", "slim_linear", "slim_linear_batched",
    "slim_adapter_codes_bytes", "slim_adapter_scales_bytes", "slim_pack_adapter",
    "slim_linear_qa_workspace_bytes", "slim_linear_qa",
    "slim_transposed_values_bytes", "slim_transposed_meta_bytes", "slim_pack_transposed",
    "slim_linear_giveups", "slim_set_wait_limit", "slim_linear_noalloc",
    "slim_quantize_input", "slim_linear_a8_workspace_bytes", "slim_linear_a8",
    "slim_pack_hybrid", "slim_linear_hybrid",
    "slim_kv_append", "slim_kv_copy_pages", "slim_attention_workspace_bytes",
    "slim_attention_decode", "slim_attention_prefill",
    "slim_rope", "slim_kv_append_rope", "slim_q4_page_bytes", "slim_kv_append_q4", "slim_kv_read_q4",
    "slim_attention_decode_q4", "slim_attention_prefill_q4",
)

_lib = None


class Rotation(ctypes.Structure):
    """slim_rotation."""
    _fields_ = [("freqs", ctypes.c_void_p), ("rot_dim", ctypes.c_int64), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_double)]


class SlimError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"status {status}: {detail}")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libslim.so once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_int4_gemm_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    i64, sz, vp = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    lib.slim_status_string.restype = ctypes.c_char_p
    lib.slim_status_string.argtypes = [ctypes.c_int]
    lib.slim_last_error.restype = ctypes.c_char_p
    lib.slim_last_error.argtypes = []
    lib.slim_version.restype = ctypes.c_int
    for f in ("slim_values_bytes", "slim_meta_bytes"):
        getattr(lib, f).restype = sz
        getattr(lib, f).argtypes = [i64, i64]
    lib.slim_scales_bytes.restype = sz
    lib.slim_scales_bytes.argtypes = [i64, i64, i64]
    lib.slim_pack.restype = ctypes.c_int
    lib.slim_pack.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp]
    lib.slim_linear_workspace_bytes.restype = sz
    lib.slim_linear_workspace_bytes.argtypes = [i64, i64, i64, i64]
    lib.slim_linear.restype = ctypes.c_int
    lib.slim_linear.argtypes = [vp, i64, i64, i64, vp, vp, vp, i64, vp, vp, i64, vp, vp, sz, vp]
    lib.slim_linear_batched.restype = ctypes.c_int
    lib.slim_linear_batched.argtypes = [i64, i64, i64, i64, i64, i64,
                                        vp, i64, vp, i64, vp, i64, vp, i64,
                                        vp, i64, vp, i64, vp, i64, vp, sz, vp]
    lib.slim_adapter_codes_bytes.restype = sz
    lib.slim_adapter_codes_bytes.argtypes = [i64, i64]
    lib.slim_adapter_scales_bytes.restype = sz
    lib.slim_adapter_scales_bytes.argtypes = [i64, i64, i64]
    lib.slim_pack_adapter.restype = ctypes.c_int
    lib.slim_pack_adapter.argtypes = [vp, i64, i64, i64, vp, vp, vp]
    lib.slim_linear_qa_workspace_bytes.restype = sz
    lib.slim_linear_qa_workspace_bytes.argtypes = [i64, i64, i64, i64]
    lib.slim_linear_qa.restype = ctypes.c_int
    lib.slim_linear_qa.argtypes = [vp, i64, i64, i64, vp, vp, vp, i64, vp, vp, vp, vp, i64, vp, vp, sz, vp]
    lib.slim_transposed_values_bytes.restype = sz
    lib.slim_transposed_values_bytes.argtypes = [i64, i64]
    lib.slim_transposed_meta_bytes.restype = sz
    lib.slim_transposed_meta_bytes.argtypes = [i64, i64]
    lib.slim_pack_transposed.restype = ctypes.c_int
    lib.slim_pack_transposed.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp]
    lib.slim_linear_giveups.restype = ctypes.c_int
    lib.slim_linear_giveups.argtypes = [vp, ctypes.c_int, ctypes.POINTER(ctypes.c_uint64), vp]
    lib.slim_set_wait_limit.restype = i64
    lib.slim_set_wait_limit.argtypes = [i64]
    lib.slim_quantize_input.restype = ctypes.c_int
    lib.slim_quantize_input.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.slim_linear_a8_workspace_bytes.restype = sz
    lib.slim_linear_a8_workspace_bytes.argtypes = [i64, i64, i64, i64]
    lib.slim_linear_a8.restype = ctypes.c_int
    lib.slim_linear_a8.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, i64, vp, vp, i64, vp, vp, sz, vp]
    lib.slim_pack_hybrid.restype = ctypes.c_int
    lib.slim_pack_hybrid.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.slim_linear_hybrid.restype = ctypes.c_int
    lib.slim_linear_hybrid.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp, vp, i64, vp, vp, sz, vp]
    lib.slim_linear_noalloc.restype = ctypes.c_int
    lib.slim_linear_noalloc.argtypes = [vp, i64, i64, i64, vp, vp, vp, i64, vp, vp, i64, vp, vp]
    i32, f32 = ctypes.c_int, ctypes.c_float
    lib.slim_kv_append.restype = ctypes.c_int
    lib.slim_kv_append.argtypes = [vp, i64, vp, i64, i64, i64, i64, i64, i32, vp, i64, vp, vp, vp, vp, i64, i64, vp]
    lib.slim_kv_copy_pages.restype = ctypes.c_int
    lib.slim_kv_copy_pages.argtypes = [vp, vp, i64, i64, i64, vp, vp, i64, vp]
    lib.slim_attention_workspace_bytes.restype = sz
    lib.slim_attention_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    lib.slim_attention_decode.restype = ctypes.c_int
    lib.slim_attention_decode.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, i32, vp, vp, i64, i64, vp, i64, vp,
                                          i64, i64, i64, f32, vp, sz, vp]
    lib.slim_attention_prefill.restype = ctypes.c_int
    lib.slim_attention_prefill.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, i64, i32, vp, vp, i64, i64, vp,
                                           i64, vp, vp, i64, i64, i64, f32, vp, sz, vp]
    rotation = ctypes.POINTER(Rotation)
    lib.slim_rope.restype = ctypes.c_int
    lib.slim_rope.argtypes = [vp, i64, vp, i64, i64, i64, i64, i32, vp, rotation, vp]
    lib.slim_q4_page_bytes.restype = sz
    lib.slim_q4_page_bytes.argtypes = [i64, i64, i64]
    for f in ("slim_kv_append_rope", "slim_kv_append_q4"):
        getattr(lib, f).restype = ctypes.c_int
        getattr(lib, f).argtypes = [vp, i64, vp, i64, i64, vp, i64, vp, i64, i64, i64, i64, i64, i32, vp, i64, vp, vp, vp,
                                    vp, i64, i64, rotation, vp]
    lib.slim_kv_read_q4.restype = ctypes.c_int
    lib.slim_kv_read_q4.argtypes = lib.slim_kv_append.argtypes
    lib.slim_attention_decode_q4.restype = ctypes.c_int
    lib.slim_attention_decode_q4.argtypes = lib.slim_attention_decode.argtypes
    lib.slim_attention_prefill_q4.restype = ctypes.c_int
    lib.slim_attention_prefill_q4.argtypes = lib.slim_attention_prefill.argtypes
    _lib = lib
    return lib


def _check(status: int):
    if status != SLIM_OK:
        lib = load()
        raise SlimError(status, f"{lib.slim_status_string(status).decode()} — {lib.slim_last_error().decode()}")


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError("tensors must live on the GPU (a ROCm 'cuda' device)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ----------------------------------------------------------- raw ABI calls
def slim_values_bytes(N: int, K: int) -> int:
    return load().slim_values_bytes(N, K)


def slim_meta_bytes(N: int, K: int) -> int:
    return load().slim_meta_bytes(N, K)


def slim_scales_bytes(N: int, K: int, group: int = 128) -> int:
    return load().slim_scales_bytes(N, K, group)


def slim_linear_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return load().slim_linear_workspace_bytes(M, N, K, r)


def slim_pack(W, values, meta, scales, group: int = 128, stream=None) -> None:
    N, K = W.shape
    _check(load().slim_pack(_ptr(W), N, K, group, _ptr(values), _ptr(meta), _ptr(scales), _stream(stream)))


def slim_linear(X, values, meta, scales, Lt, Rt, Y, workspace, group: int = 128, stream=None) -> None:
    """Lt = L^T [r, K] and Rt = R^T [N, r] (fp16); None for no adapter."""
    M, K = X.shape
    N = Y.shape[1]
    r = 0 if Lt is None else Lt.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().slim_linear(_ptr(X), M, N, K, _ptr(values), _ptr(meta), _ptr(scales), group,
                              _ptr(Lt), _ptr(Rt), r, _ptr(Y), _ptr(workspace), ws_bytes, _stream(stream)))


def slim_linear_batched(batch, M, N, K, r, X, stride_X, values, stride_values, meta, stride_meta,
                        scales, stride_scales, Lt, stride_Lt, Rt, stride_Rt, Y, stride_Y, workspace,
                        group: int = 128, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().slim_linear_batched(batch, M, N, K, r, group,
                                      _ptr(X), stride_X, _ptr(values), stride_values,
                                      _ptr(meta), stride_meta, _ptr(scales), stride_scales,
                                      _ptr(Lt), stride_Lt, _ptr(Rt), stride_Rt, _ptr(Y), stride_Y,
                                      _ptr(workspace), ws_bytes, _stream(stream)))


def slim_adapter_codes_bytes(rows: int, cols: int) -> int:
    return load().slim_adapter_codes_bytes(rows, cols)


def slim_adapter_scales_bytes(rows: int, cols: int, group: int) -> int:
    return load().slim_adapter_scales_bytes(rows, cols, group)


def slim_linear_qa_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return load().slim_linear_qa_workspace_bytes(M, N, K, r)


def slim_pack_adapter(A, codes, scales, group: int, stream=None) -> None:
    """A: fp32 factor [rows, cols] stored output-major (Lt or Rt)."""
    rows, cols = A.shape
    _check(load().slim_pack_adapter(_ptr(A), rows, cols, group, _ptr(codes), _ptr(scales), _stream(stream)))


def slim_linear_qa(X, values, meta, scales, Lq, Ls, Rq, Rs, r, Y, workspace, group: int = 128, stream=None) -> None:
    M, K = X.shape
    N = Y.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().slim_linear_qa(_ptr(X), M, N, K, _ptr(values), _ptr(meta), _ptr(scales), group,
                                 _ptr(Lq), _ptr(Ls), _ptr(Rq), _ptr(Rs), r, _ptr(Y), _ptr(workspace), ws_bytes,
                                 _stream(stream)))


def slim_transposed_values_bytes(N: int, K: int) -> int:
    return load().slim_transposed_values_bytes(N, K)


def slim_transposed_meta_bytes(N: int, K: int) -> int:
    return load().slim_transposed_meta_bytes(N, K)


def slim_pack_transposed(values, meta, scales, N: int, K: int, tvalues, tmeta, group: int = 128,
                         stream=None) -> None:
    """Double-pruned transpose of a packed W [N, K]: tvalues fp16 [K, N/2],
    tmeta uint16 [K, N/16] (int16 tensors hold the bit patterns)."""
    _check(load().slim_pack_transposed(_ptr(values), _ptr(meta), _ptr(scales), N, K, group, _ptr(tvalues),
                                       _ptr(tmeta), _stream(stream)))


def slim_linear_giveups(workspace, reset: bool = False, stream=None) -> int:
    """Workgroups of the one-launch decode path that gave up their bounded
    wait on this workspace (synchronises the stream)."""
    n = ctypes.c_uint64(0)
    _check(load().slim_linear_giveups(_ptr(workspace), 1 if reset else 0, ctypes.byref(n), _stream(stream)))
    return int(n.value)


def slim_set_wait_limit(limit: int) -> int:
    """Poll passes before a one-launch decode workgroup gives up (0: at once,
    negative: the default).  Returns the previous limit."""
    return int(load().slim_set_wait_limit(limit))


def slim_linear_noalloc(X, values, meta, scales, Lt, Rt, Y, group: int = 128, stream=None) -> None:
    """slim_linear with the library's own per-GPU scratch (no workspace)."""
    M, K = X.shape
    N = Y.shape[1]
    r = 0 if Lt is None else Lt.shape[0]
    _check(load().slim_linear_noalloc(_ptr(X), M, N, K, _ptr(values), _ptr(meta), _ptr(scales), group,
                                      _ptr(Lt), _ptr(Rt), r, _ptr(Y), _stream(stream)))


def slim_quantize_input(X, q, s, stream=None) -> None:
    """Per-token int8 quantisation of fp16 X [M, K] into q (int8 [M, K]) and s (fp16 [M])."""
    M, K = X.shape
    _check(load().slim_quantize_input(_ptr(X), M, K, _ptr(q), _ptr(s), _stream(stream)))


def slim_linear_a8_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return load().slim_linear_a8_workspace_bytes(M, N, K, r)


def slim_linear_a8(qx, sx, values, meta, scales, Lt, Rt, Y, workspace, group: int = 128, stream=None) -> None:
    """The layer on an 8-bit input: qx int8 [M, K], sx fp16 [M]."""
    M, K = qx.shape
    N = Y.shape[1]
    r = 0 if Lt is None else Lt.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().slim_linear_a8(_ptr(qx), _ptr(sx), M, N, K, _ptr(values), _ptr(meta), _ptr(scales), group,
                                 _ptr(Lt), _ptr(Rt), r, _ptr(Y), _ptr(workspace), ws_bytes, _stream(stream)))


def slim_pack_hybrid(W, dense, values, meta, scales, dvalues, group: int = 128, stream=None) -> None:
    """Hybrid dense / 2:4 pack; dense: int32 [ceil(N/16), K/128] tile flags."""
    N, K = W.shape
    _check(load().slim_pack_hybrid(_ptr(W), N, K, group, _ptr(dense), _ptr(values), _ptr(meta), _ptr(scales),
                                   _ptr(dvalues), _stream(stream)))


def slim_linear_hybrid(X, values, meta, scales, dvalues, dense, Lt, Rt, Y, workspace, group: int = 128,
                       stream=None) -> None:
    M, K = X.shape
    N = Y.shape[1]
    r = 0 if Lt is None else Lt.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().slim_linear_hybrid(_ptr(X), M, N, K, _ptr(values), _ptr(meta), _ptr(scales), _ptr(dvalues),
                                     _ptr(dense), group, _ptr(Lt), _ptr(Rt), r, _ptr(Y), _ptr(workspace), ws_bytes,
                                     _stream(stream)))


# ------------------------------------- paged key-value cache and attention
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_PAGE_TYPES = (*_DTYPES, torch.uint8)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


# (Each attribute of a tensor costs some 50 ns, a call's checks as much as its
# launch: every one is read once.)
def _rows(name, t, heads, dim, dtype, device):
    """(pointer, row stride, tokens, heads) of a [tokens, heads, dim] tensor whose
    rows are dense; the rows themselves may lie apart (a slice of a joint
    array).  heads None: any number."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {dim}], got {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    tokens, heads, _ = shape
    sr, sh, sd = t.stride()
    if sd != 1 or (sh != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), sr if tokens > 1 else heads * dim, tokens, heads


def _ints(name, t, device, dims):
    """Pointer and shape."""
    shape = t.shape
    if t.dtype is not torch.int32 or len(shape) != dims or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dims}-dimensional int32 tensor on {device}")
    return t.data_ptr(), shape


def _pools(kpool, vpool, dims, dtypes=_DTYPES):
    """Device, shape, type and pointers of a pair of pools."""
    if not kpool.is_cuda:
        raise ValueError("tensors must live on the GPU (a ROCm 'cuda' device)")
    device, shape, dtype = kpool.device, kpool.shape, kpool.dtype
    if dtype not in dtypes:
        raise TypeError("the pools must be float16 or bfloat16" if dtypes is _DTYPES else
                        "the pools must be float16, bfloat16 or uint8 (pages of 4 bits)")
    if len(shape) not in dims or shape != vpool.shape or dtype is not vpool.dtype or device != vpool.device:
        raise ValueError(f"the pools must be two {' or '.join(map(str, dims))}-dimensional tensors of one shape, type "
                         "and device")
    if not (kpool.is_contiguous() and vpool.is_contiguous()):
        raise ValueError("the pools must be contiguous")
    return device, shape, dtype, kpool.data_ptr(), vpool.data_ptr()


def _stream_on(stream, device):
    """The HIP stream of a call on `device`, and a check that launches go there."""
    if device.index != _current_device():
        raise ValueError(f"the current device must be the tensors' {device}")
    if stream is not None:
        return stream.cuda_stream
    return _current_stream(device)


def _current_stream(device):
    """Handle of the device's current stream."""
    # (The public way to it costs as much as the launch.)
    return _raw_stream(device.index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream


def _batch(table, lens, starts, tokens, device):
    """Pointers of table, lens and starts, the number of sequences and the table's width."""
    p_table, (rows, width) = _ints("table", table, device, 2)
    p_lens, (seqs,) = _ints("lens", lens, device, 1)
    if rows != seqs:
        raise ValueError(f"table has {rows} rows for {seqs} sequences")
    if starts is None:
        if tokens != seqs:
            raise ValueError(f"{tokens} new tokens for {seqs} sequences without starts")
        return p_table, p_lens, None, seqs, width
    p_starts, (bounds,) = _ints("starts", starts, device, 1)
    if bounds != seqs + 1:
        raise ValueError(f"starts must hold {seqs + 1} values, got {bounds}")
    return p_table, p_lens, p_starts, seqs, width


def slim_kv_append(K, V, kpool, vpool, table, lens, starts=None, stream=None) -> None:
    """K, V [tokens, kv_heads, head_dim] to the pages of their positions; pools [pages, kv_heads, page_size, head_dim]."""
    dev, (pages, heads, page, dim), dtype, pkp, pvp = _pools(kpool, vpool, (4,))
    pk, sk, tokens, _ = _rows("K", K, heads, dim, dtype, dev)
    pv, sv, v_tokens, _ = _rows("V", V, heads, dim, dtype, dev)
    if v_tokens != tokens:
        raise ValueError(f"K has {tokens} rows and V {v_tokens}")
    pt, pl, ps, seqs, width = _batch(table, lens, starts, tokens, dev)
    _check(load().slim_kv_append(pk, sk, pv, sv, tokens, seqs, heads, dim, _DTYPES[dtype], pt, width, pl, ps, pkp, pvp,
                                 pages, page, _stream_on(stream, dev)))


def _q4_pools(kpool, vpool):
    """Device, (pages, kv_heads, page_size, head_dim) and pointers of a pair of 4-bit pools."""
    if not kpool.is_cuda:
        raise ValueError("tensors must live on the GPU (a ROCm 'cuda' device)")
    device, shape = kpool.device, kpool.shape
    if kpool.dtype is not torch.uint8 or vpool.dtype is not torch.uint8:
        raise TypeError("the pools must be uint8 [pages, kv_heads, page_size, head_dim * 17 / 32]")
    if len(shape) != 4 or shape != vpool.shape or device != vpool.device:
        raise ValueError("the pools must be two 4-dimensional tensors of one shape and device")
    if not (kpool.is_contiguous() and vpool.is_contiguous()):
        raise ValueError("the pools must be contiguous")
    pages, heads, page, row = shape
    if row % 17:
        raise ValueError(f"a row of a 4-bit pool holds head_dim * 17 / 32 bytes, not {row}")
    return device, (pages, heads, page, row // 17 * 32), kpool.data_ptr(), vpool.data_ptr()


def slim_kv_copy_pages(kpool, vpool, src, dst, stream=None) -> None:
    """Pages src[i] to dst[i] of every layer; pools [layers, pages, ...] or one layer's
    [pages, kv_heads, page_size, head_dim] (uint8: 4-bit pages)."""
    dev, shape, dtype, pkp, pvp = _pools(kpool, vpool, (4, 5), _PAGE_TYPES)
    layers = shape[0] if len(shape) == 5 else 1
    pages, heads, page, dim = shape[-4:]
    (ps, (count,)), (pd, (to,)) = _ints("src", src, dev, 1), _ints("dst", dst, dev, 1)
    if count != to:
        raise ValueError(f"{count} sources and {to} destinations")
    _check(load().slim_kv_copy_pages(pkp, pvp, layers, pages, heads * page * dim * dtype.itemsize, ps, pd, count,
                                     _stream_on(stream, dev)))


def slim_attention_workspace_bytes(tokens: int, seqs: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return load().slim_attention_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim)


def _attention_args(Q, O, lse, kpool, vpool, table, lens, starts, workspace, max_len, window, sinks, scale, stream, q4=False):
    """What both attention calls pass on: before seqs' place, from it to lens',
    and after.  max_len None: the table's capacity; scale None: 1 / sqrt(head_dim)."""
    if q4:
        dev, (pages, kv_heads, page, dim), pk, pv = _q4_pools(kpool, vpool)
        dtype = _half(Q, "Q")
    else:
        dev, (pages, kv_heads, page, dim), dtype, pk, pv = _pools(kpool, vpool, (4,))
    pq, sq, tokens, q_heads = _rows("Q", Q, None, dim, dtype, dev)
    po, so, o_tokens, _ = _rows("O", O, q_heads, dim, dtype, dev)
    if o_tokens != tokens:
        raise ValueError(f"Q has {tokens} rows and O {o_tokens}")
    p_lse = None
    if lse is not None:
        if lse.dtype != torch.float32 or lse.shape != (tokens, q_heads) or not lse.is_contiguous() or lse.device != dev:
            raise ValueError(f"lse must be a contiguous float32 [{tokens}, {q_heads}] tensor on {dev}")
        p_lse = lse.data_ptr()
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on {dev}")
    pt, pl, ps, seqs, width = _batch(table, lens, starts, tokens, dev)
    if max_len is None:
        max_len = width * page
    if scale is None:
        scale = dim ** -0.5
    return ((pq, sq, po, so, p_lse), tokens, (seqs, q_heads, kv_heads, dim, _DTYPES[dtype], pk, pv, pages, page, pt, width,
            pl), ps, (max_len, window, sinks, scale, workspace.data_ptr(), workspace.nbytes, _stream_on(stream, dev)))


def slim_attention_decode(Q, O, kpool, vpool, table, lens, workspace, max_len: int, window: int = 0, sinks: int = 0,
                          scale: float = 1.0, lse=None, stream=None) -> None:
    """Attention of one new token per sequence: Q, O [seqs, q_heads, head_dim]."""
    rows, _, cache, _, rest = _attention_args(Q, O, lse, kpool, vpool, table, lens, None, workspace, max_len, window,
                                              sinks, scale, stream)
    _check(load().slim_attention_decode(*rows, *cache, *rest))


def slim_attention_prefill(Q, O, kpool, vpool, table, lens, starts, workspace, max_len: int, window: int = 0,
                           sinks: int = 0, scale: float = 1.0, lse=None, stream=None) -> None:
    """Attention of any number of new tokens per sequence: Q, O [tokens, q_heads, head_dim]."""
    rows, tokens, cache, ps, rest = _attention_args(Q, O, lse, kpool, vpool, table, lens, starts, workspace, max_len,
                                                    window, sinks, scale, stream)
    _check(load().slim_attention_prefill(*rows, tokens, *cache, ps, *rest))


def _half(t, name):
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return t.dtype


def _rotation(rope, device, handle, stream):
    """slim_rotation of a Rope (kept by it) for a call on stream `handle` (`stream`, or the current one if None);
    None of None."""
    if rope is None:
        return None
    freqs = rope.freqs
    if freqs.device != device:
        raise ValueError(f"the rotation must be on {device}, got {freqs.device}")
    if handle != rope.made_on:
        # It may be let go before that stream has read its frequencies.
        freqs.record_stream(torch.cuda.current_stream(device) if stream is None else stream)
    return rope.params


def slim_rope(X, Y, positions, rope, stream=None) -> None:
    """X, Y [tokens, heads, head_dim], positions int32 [tokens], rope: a Rope."""
    if not X.is_cuda:
        raise ValueError("tensors must live on the GPU (a ROCm 'cuda' device)")
    if X.dim() != 3:
        raise ValueError(f"X must be [tokens, heads, head_dim], got {tuple(X.shape)}")
    dev, dtype = X.device, _half(X, "X")
    px, sx, tokens, heads = _rows("X", X, None, X.shape[2], dtype, dev)
    py, sy, y_tokens, _ = _rows("Y", Y, heads, X.shape[2], dtype, dev)
    pp, (count,) = _ints("positions", positions, dev, 1)
    if y_tokens != tokens or count != tokens:
        raise ValueError(f"X has {tokens} rows, Y {y_tokens}, and there are {count} positions")
    handle = _stream_on(stream, dev)
    _check(load().slim_rope(px, sx, py, sy, tokens, heads, X.shape[2], _DTYPES[dtype], pp,
                            _rotation(rope, dev, handle, stream), handle))


def _append_args(K, V, heads, dim, dtype, dev):
    pk, sk, tokens, _ = _rows("K", K, heads, dim, dtype, dev)
    pv, sv, v_tokens, _ = _rows("V", V, heads, dim, dtype, dev)
    if v_tokens != tokens:
        raise ValueError(f"K has {tokens} rows and V {v_tokens}")
    return pk, sk, pv, sv, tokens


def _append(call, Q, Qout, K, V, pkp, pvp, pages, heads, page, dim, dtype, dev, table, lens, rope, starts, stream):
    pk, sk, pv, sv, tokens = _append_args(K, V, heads, dim, dtype, dev)
    queries = (None, 0, None, 0, 0)
    if (Q is None) != (Qout is None):
        raise ValueError("Q and Qout must both be given, or neither")
    if Q is not None:
        pq, sq, q_tokens, q_heads = _rows("Q", Q, None, dim, dtype, dev)
        po, so, o_tokens, _ = _rows("Qout", Qout, q_heads, dim, dtype, dev)
        if q_tokens != tokens or o_tokens != tokens:
            raise ValueError(f"K has {tokens} rows, Q {q_tokens} and Qout {o_tokens}")
        queries = (pq, sq, po, so, q_heads)
    pt, pl, ps, seqs, width = _batch(table, lens, starts, tokens, dev)
    handle = _stream_on(stream, dev)
    _check(call(*queries, pk, sk, pv, sv, tokens, seqs, heads, dim, _DTYPES[dtype], pt, width, pl, ps, pkp, pvp, pages, page,
                _rotation(rope, dev, handle, stream), handle))


def slim_kv_append_rope(Q, Qout, K, V, kpool, vpool, table, lens, rope, starts=None, stream=None) -> None:
    """slim_kv_append with the keys turned by rope, and Q [tokens, q_heads, head_dim] into Qout (or both None)."""
    dev, (pages, heads, page, dim), dtype, pkp, pvp = _pools(kpool, vpool, (4,))
    _append(load().slim_kv_append_rope, Q, Qout, K, V, pkp, pvp, pages, heads, page, dim, dtype, dev, table, lens, rope,
            starts, stream)


def slim_q4_page_bytes(kv_heads: int, page_size: int, head_dim: int) -> int:
    return load().slim_q4_page_bytes(kv_heads, page_size, head_dim)


def slim_kv_append_q4(Q, Qout, K, V, kpool, vpool, table, lens, rope=None, starts=None, stream=None) -> None:
    """slim_kv_append_rope into uint8 pools [pages, kv_heads, page_size, head_dim * 17 / 32]; rope None: keys as they are."""
    dev, (pages, heads, page, dim), pkp, pvp = _q4_pools(kpool, vpool)
    _append(load().slim_kv_append_q4, Q, Qout, K, V, pkp, pvp, pages, heads, page, dim, _half(K, "K"), dev, table, lens,
            rope, starts, stream)


def slim_kv_read_q4(K, V, kpool, vpool, table, lens, starts=None, stream=None) -> None:
    """The new tokens' keys and values from the pages to K, V [tokens, kv_heads, head_dim]."""
    dev, (pages, heads, page, dim), pkp, pvp = _q4_pools(kpool, vpool)
    dtype = _half(K, "K")
    pk, sk, pv, sv, tokens = _append_args(K, V, heads, dim, dtype, dev)
    pt, pl, ps, seqs, width = _batch(table, lens, starts, tokens, dev)
    _check(load().slim_kv_read_q4(pk, sk, pv, sv, tokens, seqs, heads, dim, _DTYPES[dtype], pt, width, pl, ps, pkp, pvp,
                                  pages, page, _stream_on(stream, dev)))


def slim_attention_decode_q4(Q, O, kpool, vpool, table, lens, workspace, max_len: int, window: int = 0, sinks: int = 0,
                             scale: float = 1.0, lse=None, stream=None) -> None:
    """slim_attention_decode over 4-bit pools."""
    rows, _, cache, _, rest = _attention_args(Q, O, lse, kpool, vpool, table, lens, None, workspace, max_len, window,
                                              sinks, scale, stream, True)
    _check(load().slim_attention_decode_q4(*rows, *cache, *rest))


def slim_attention_prefill_q4(Q, O, kpool, vpool, table, lens, starts, workspace, max_len: int, window: int = 0,
                              sinks: int = 0, scale: float = 1.0, lse=None, stream=None) -> None:
    """slim_attention_prefill over 4-bit pools."""
    rows, tokens, cache, ps, rest = _attention_args(Q, O, lse, kpool, vpool, table, lens, starts, workspace, max_len,
                                                    window, sinks, scale, stream, True)
    _check(load().slim_attention_prefill_q4(*rows, tokens, *cache, ps, *rest))
