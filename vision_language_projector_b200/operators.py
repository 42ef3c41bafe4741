"""Operators around the projector's training step: token-embedding lookup and the
gradient of its table, layer norm and its gradients, gradient clipping by the global norm.

Argument marshalling for ``vlproj_embed``, ``vlproj_embed_backward``,
``vlproj_layernorm``, ``vlproj_layernorm_backward`` and ``vlproj_clip_grads`` of
``include/vlproj.h``, which holds their formulas. Tensors are bf16, fp16 or fp32 CUDA
tensors on the current device; every output is passed in. Matrices are contiguous (their
leading axes taken together are the rows) or two-dimensional with rows of their own
distance. A workspace comes from torch's allocator, on the stream of the call, unless one
is passed (a contiguous uint8 tensor on a multiple of 256 bytes, as large as the
``*_workspace`` function says, and of this call alone while it runs).

Calls raise :class:`VlprojError` on an argument the library cannot take and return the
status code; with ``check=False`` they only return it.
"""
from __future__ import annotations

import ctypes
from array import array
from typing import Optional

from . import OK, VlprojError, _arg_error, _lib

BF16, F32, F16 = 0, 1, 2
NO_TOKEN = -(1 << 63)
CLIP_FEW_TENSORS, CLIP_FEW_ELEMENTS = 16, 256 * 1024      # clip_grads needs no workspace up to these

_I32, _I64, _P, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class EmbedArgs(ctypes.Structure):
    """Mirror of ``vlproj_embed_args``."""
    _fields_ = [("input_ids", _P), ("n_ids", _I64), ("image_token_id", _I64), ("table", _P), ("vocab", _I64),
                ("table_ld", _I64), ("out", _P), ("out_ld", _I64), ("N", _I64), ("scale", _F), ("table_type", _I32),
                ("out_type", _I32), ("status", _P)]


class EmbedBackwardArgs(ctypes.Structure):
    """Mirror of ``vlproj_embed_backward_args``."""
    _fields_ = [("input_ids", _P), ("n_ids", _I64), ("image_token_id", _I64), ("d_out", _P), ("d_out_ld", _I64),
                ("d_table", _P), ("d_table_ld", _I64), ("vocab", _I64), ("N", _I64), ("scale", _F),
                ("d_out_type", _I32), ("accumulate", _I32), ("status", _P), ("workspace", _P),
                ("workspace_bytes", _I64)]


class LayernormArgs(ctypes.Structure):
    """Mirror of ``vlproj_layernorm_args``."""
    _fields_ = [("x", _P), ("x_ld", _I64), ("y", _P), ("y_ld", _I64), ("rows", _I64), ("C", _I64), ("gamma", _P),
                ("beta", _P), ("mean", _P), ("rstd", _P), ("eps", _F), ("x_type", _I32), ("y_type", _I32)]


class LayernormBackwardArgs(ctypes.Structure):
    """Mirror of ``vlproj_layernorm_backward_args``."""
    _fields_ = [("x", _P), ("x_ld", _I64), ("mean", _P), ("rstd", _P), ("d_y", _P), ("d_y_ld", _I64), ("gamma", _P),
                ("d_x", _P), ("d_x_ld", _I64), ("d_gamma", _P), ("d_beta", _P), ("rows", _I64), ("C", _I64),
                ("x_type", _I32), ("y_type", _I32), ("workspace", _P), ("workspace_bytes", _I64)]


class ClipGradsArgs(ctypes.Structure):
    """Mirror of ``vlproj_clip_grads_args``."""
    _fields_ = [("n", _I32), ("grads", _P), ("out", _P), ("numel", _P), ("type", _P), ("max_norm", ctypes.c_double),
                ("norm", _P), ("workspace", _P), ("workspace_bytes", _I64)]


def _bind() -> None:
    for name, args in (("embed", EmbedArgs), ("embed_backward", EmbedBackwardArgs), ("layernorm", LayernormArgs),
                       ("layernorm_backward", LayernormBackwardArgs), ("clip_grads", ClipGradsArgs)):
        fn = getattr(_lib, "vlproj_" + name)
        fn.argtypes, fn.restype = [ctypes.POINTER(args), _P], ctypes.c_int
    for name, args in (("embed_backward", [_I64, _I64]), ("layernorm_backward", [_I64, _I64]), ("clip_grads", [_I32])):
        fn = getattr(_lib, f"vlproj_{name}_workspace")
        fn.argtypes, fn.restype = args, _I64


_bind()

# torch, its element types and its two queries that a call makes, on first use: this module
# is imported before torch where only the host functions are wanted
_torch = _types = _current_device = _current_stream = None


def _use_torch() -> None:
    global _torch, _types, _current_device, _current_stream
    import torch
    _types = {torch.bfloat16: BF16, torch.float32: F32, torch.float16: F16}
    # what torch.cuda.current_device() and current_stream().cuda_stream return, without the
    # objects around them: a small call spends as long in this module as on the GPU
    _current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _torch = torch


def _device() -> int:
    """The current device; every tensor of a call has to be on it."""
    if _torch is None:
        _use_torch()
    return _current_device()


def _on(t, name: str, dev: int) -> None:
    try:
        d = t.get_device()                    # -1 on the host
    except AttributeError:
        raise _arg_error(name, f"a CUDA tensor is required, got {type(t).__name__}") from None
    if d != dev:
        if d < 0:
            raise _arg_error(name, f"a CUDA tensor is required, got one on {t.device}")
        raise _arg_error(name, f"a tensor on {t.device}, the current device is cuda:{dev}")


def _type(t, name: str) -> int:
    code = _types.get(t.dtype)
    if code is None:
        raise _arg_error(name, f"{t.dtype} is not bf16, fp16 or fp32")
    return code


def _vector(t, name: str, dev: int, dtype, numel: int) -> Optional[int]:
    if t is None:
        return None
    _on(t, name, dev)
    if t.dtype != dtype or t.numel() != numel or not t.is_contiguous():
        raise _arg_error(name, f"{numel} contiguous elements of {dtype} are required, got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def _matrix(t, name: str, dev: int):
    """(address, rows, row length, row distance) of a matrix."""
    _on(t, name, dev)
    shape = t.shape
    n = shape[-1] if shape else 0
    if n < 1:
        raise _arg_error(name, f"rows of one element or more are required, got {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), t.numel() // n, n, n
    if len(shape) == 2 and (t.stride(1) == 1 or n == 1):
        ld = t.stride(0) if shape[0] > 1 else n
        if ld >= n:
            return t.data_ptr(), shape[0], n, ld
    raise _arg_error(name, f"rows with adjacent elements that do not overlap are required, got strides {t.stride()}")


def _stream(stream, dev: int) -> int:
    if stream is None:
        return _current_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _workspace(given, nbytes: int, stream, dev: int):
    """(tensor to keep until the launch, address, bytes). Memory taken here belongs to the
    call's stream, so the allocator hands it out again only behind the call."""
    if nbytes < 0:
        raise VlprojError(nbytes, "workspace size")
    torch = _torch
    if nbytes == 0:
        return None, None, 0
    if given is not None:
        _on(given, "workspace", dev)
        if given.dtype != torch.uint8 or not given.is_contiguous() or given.numel() < nbytes:
            raise _arg_error("workspace", f"{nbytes} contiguous bytes are required, got {given.numel()} of {given.dtype}")
        return given, given.data_ptr(), given.numel()
    if stream is None:
        w = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        s = stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s) if s else torch.cuda.default_stream()
        with torch.cuda.stream(s):
            w = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return w, w.data_ptr(), nbytes


def _finish(rc: int, what: str, check: bool) -> int:
    if check and rc != OK:
        raise VlprojError(rc, what)
    return rc


def _reject(e: VlprojError, check: bool) -> int:
    if check:
        raise e
    return e.code


def _ids(t, dev: int):
    _on(t, "input_ids", dev)
    if t.dtype != _torch.int64 or not t.is_contiguous():
        raise _arg_error("input_ids", f"contiguous int64 ids are required, got {t.dtype}")
    return t.data_ptr(), t.numel()


def _token(image_token_id) -> int:
    if image_token_id is None:
        return NO_TOKEN
    t = int(image_token_id)
    if not -(1 << 63) <= t < 1 << 63:                    # ctypes would keep its low 64 bits
        raise _arg_error("image_token_id", f"{t} is not an int64")
    return t


def embed(input_ids, table, out, scale: float = 1.0, image_token_id: Optional[int] = None, status=None, stream=None,
          check: bool = True) -> int:
    """``vlproj_embed``: row i of ``out`` (n_ids, N) becomes ``scale * table[input_ids[i]]``;
    rows of ``image_token_id`` stay as they were. ``table`` (vocab, N) has out's type, or is
    fp32. An id outside the table gives a zero row and latches ERR_INVALID_ARG in
    ``status`` (int32, one element, optional)."""
    dev = _device()
    try:
        ids, n = _ids(input_ids, dev)
        pt, vocab, N, t_ld = _matrix(table, "table", dev)
        po, rows, n_out, o_ld = _matrix(out, "out", dev)
        if rows < n or n_out != N:
            raise _arg_error("out", f"({rows}, {n_out}) for {n} ids and rows of {N}")
        a = EmbedArgs(ids, n, _token(image_token_id), pt, vocab, t_ld, po, o_ld, N,
                      scale, _type(table, "table"), _type(out, "out"),
                      _vector(status, "status", dev, _torch.int32, 1))
    except VlprojError as e:
        return _reject(e, check)
    return _finish(_lib.vlproj_embed(a, _stream(stream, dev)), "vlproj_embed", check)


def embed_backward_workspace(n_ids: int, N: int) -> int:
    """Bytes of workspace ``embed_backward`` needs."""
    return _size(_lib.vlproj_embed_backward_workspace(n_ids, N), "vlproj_embed_backward_workspace")


def embed_backward(input_ids, d_out, d_table, scale: float = 1.0, image_token_id: Optional[int] = None,
                   accumulate: bool = False, status=None, workspace=None, stream=None, check: bool = True) -> int:
    """``vlproj_embed_backward``: ``d_table`` (vocab, N) fp32 becomes the gradient of the
    lookup's table for the gradient ``d_out`` (n_ids, N) of its output: per token the scaled
    sum of its rows, zeros for tokens that do not occur; ``accumulate`` adds the sums
    instead and leaves the other rows as they were."""
    dev = _device()
    try:
        ids, n = _ids(input_ids, dev)
        pd, rows, N, d_ld = _matrix(d_out, "d_out", dev)
        pt, vocab, n_t, t_ld = _matrix(d_table, "d_table", dev)
        if rows < n:
            raise _arg_error("d_out", f"{rows} rows for {n} ids")
        if n_t != N or d_table.dtype != _torch.float32:
            raise _arg_error("d_table", f"fp32 rows of {N} are required, got {n_t} of {d_table.dtype}")
        w, pw, nw = _workspace(workspace, _lib.vlproj_embed_backward_workspace(n, N), stream, dev)
        a = EmbedBackwardArgs(ids, n, _token(image_token_id), pd, d_ld, pt, t_ld,
                              vocab, N, scale, _type(d_out, "d_out"), int(accumulate),
                              _vector(status, "status", dev, _torch.int32, 1), pw, nw)
    except VlprojError as e:
        return _reject(e, check)
    return _finish(_lib.vlproj_embed_backward(a, _stream(stream, dev)), "vlproj_embed_backward", check)


def layernorm(x, y, gamma=None, beta=None, eps: float = 1e-5, mean=None, rstd=None, stream=None,
              check: bool = True) -> int:
    """``vlproj_layernorm``: ``y`` becomes the layer norm of ``x`` over its last axis, scaled
    by ``gamma`` and shifted by ``beta`` (fp32, optional); ``mean`` and ``rstd`` (fp32, one per
    row, optional) receive the statistics ``layernorm_backward`` reads. ``y`` has x's type, or
    x is fp32."""
    dev = _device()
    try:
        f32 = _torch.float32
        px, rows, C, x_ld = _matrix(x, "x", dev)
        py, y_rows, y_C, y_ld = _matrix(y, "y", dev)
        if y_rows != rows or y_C != C:
            raise _arg_error("y", f"({y_rows}, {y_C}) for rows ({rows}, {C})")
        a = LayernormArgs(px, x_ld, py, y_ld, rows, C, _vector(gamma, "gamma", dev, f32, C),
                          _vector(beta, "beta", dev, f32, C), _vector(mean, "mean", dev, f32, rows),
                          _vector(rstd, "rstd", dev, f32, rows), eps, _type(x, "x"), _type(y, "y"))
    except VlprojError as e:
        return _reject(e, check)
    return _finish(_lib.vlproj_layernorm(a, _stream(stream, dev)), "vlproj_layernorm", check)


def layernorm_backward_workspace(rows: int, C: int) -> int:
    """Bytes of workspace ``layernorm_backward`` needs for ``d_gamma`` or ``d_beta``."""
    return _size(_lib.vlproj_layernorm_backward_workspace(rows, C), "vlproj_layernorm_backward_workspace")


def layernorm_backward(x, mean, rstd, d_y, gamma=None, d_x=None, d_gamma=None, d_beta=None, workspace=None, stream=None,
                       check: bool = True) -> int:
    """``vlproj_layernorm_backward``: gradients of ``layernorm`` for the gradient ``d_y`` of its
    output (y's type): ``d_x`` (x's type), ``d_gamma`` and ``d_beta`` (fp32), each optional and
    overwritten."""
    dev = _device()
    try:
        f32 = _torch.float32
        px, rows, C, x_ld = _matrix(x, "x", dev)
        pd, d_rows, d_C, d_ld = _matrix(d_y, "d_y", dev)
        if d_rows != rows or d_C != C:
            raise _arg_error("d_y", f"({d_rows}, {d_C}) for rows ({rows}, {C})")
        pg, g_ld = None, 0
        if d_x is not None:
            pg, g_rows, g_C, g_ld = _matrix(d_x, "d_x", dev)
            if g_rows != rows or g_C != C or d_x.dtype != x.dtype:
                raise _arg_error("d_x", f"({g_rows}, {g_C}) {d_x.dtype} for x ({rows}, {C}) {x.dtype}")
        if mean is None or rstd is None:
            raise _arg_error("mean" if mean is None else "rstd", "the forward pass's statistics are required")
        w, pw, nw = None, None, 0
        if d_gamma is not None or d_beta is not None:
            w, pw, nw = _workspace(workspace, _lib.vlproj_layernorm_backward_workspace(rows, C), stream, dev)
        a = LayernormBackwardArgs(px, x_ld, _vector(mean, "mean", dev, f32, rows), _vector(rstd, "rstd", dev, f32, rows),
                                  pd, d_ld, _vector(gamma, "gamma", dev, f32, C), pg, g_ld,
                                  _vector(d_gamma, "d_gamma", dev, f32, C), _vector(d_beta, "d_beta", dev, f32, C), rows,
                                  C, _type(x, "x"), _type(d_y, "d_y"), pw, nw)
    except VlprojError as e:
        return _reject(e, check)
    return _finish(_lib.vlproj_layernorm_backward(a, _stream(stream, dev)), "vlproj_layernorm_backward", check)


def _flat(grads) -> list:
    """The tensors of a sequence, or of a dict such as ``Projector.backward`` fills
    (entries may be lists, and None where a gradient is not wanted)."""
    got = []
    for v in (grads.values() if isinstance(grads, dict) else grads):
        if v is None:
            continue
        if v.__class__ is list or v.__class__ is tuple:
            got += [t for t in v if t is not None]
        else:
            got.append(v)
    return got


def _flat_args(ts: list, name: str, dev: int):
    """(addresses, element counts, type codes) of contiguous tensors on the device."""
    try:
        if all([t.get_device() == dev and t.is_contiguous() for t in ts]):
            return (array("q", [t.data_ptr() for t in ts]), array("q", [t.numel() for t in ts]),
                    array("i", [_types[t.dtype] for t in ts]))
    except (AttributeError, KeyError):
        pass
    for i, t in enumerate(ts):                       # which one it is
        _on(t, f"{name}[{i}]", dev)
        _type(t, f"{name}[{i}]")
        if not t.is_contiguous():
            raise _arg_error(f"{name}[{i}]", "the tensor must be contiguous")
    raise _arg_error(name, "tensors are required")


def _clip(grads, max_norm: float, norm, out, workspace, stream, check: bool) -> int:
    dev = _device()
    try:
        ts = _flat(grads)
        n = len(ts)
        ptrs, numel, types = _flat_args(ts, "grads", dev)
        p_out, outs = None, None
        if out is grads:
            p_out = ptrs.buffer_info()[0]
        elif out is not None:
            os_ = _flat(out)
            if len(os_) != n:
                raise _arg_error("out", f"{len(os_)} tensors for {n} gradients")
            outs, o_numel, o_types = _flat_args(os_, "out", dev)
            if o_numel != numel or o_types != types:
                i = next(i for i in range(n) if o_numel[i] != numel[i] or o_types[i] != types[i])
                raise _arg_error(f"out[{i}]", f"{numel[i]} elements of {ts[i].dtype} are required, got {o_numel[i]} of "
                                              f"{os_[i].dtype}")
            p_out = outs.buffer_info()[0]
        pn = _vector(norm, "norm", dev, _torch.float32, 1)
        if n == 0 and pn is None:
            return OK
        w, pw, nw = None, None, 0
        if workspace is not None or n > CLIP_FEW_TENSORS or sum(numel) > CLIP_FEW_ELEMENTS:
            w, pw, nw = _workspace(workspace, _lib.vlproj_clip_grads_workspace(n), stream, dev)
        a = ClipGradsArgs(n, ptrs.buffer_info()[0], p_out, numel.buffer_info()[0], types.buffer_info()[0], max_norm, pn,
                          pw, nw)
    except VlprojError as e:
        return _reject(e, check)
    # the library reads the four arrays before it returns
    return _finish(_lib.vlproj_clip_grads(a, _stream(stream, dev)), "vlproj_clip_grads", check)


def grad_norm(grads, norm, workspace=None, stream=None, check: bool = True) -> int:
    """The global 2-norm of all tensors of ``grads`` (a sequence, or a dict as
    ``Projector.backward`` fills) into ``norm`` (fp32, one element)."""
    if norm is None:
        return _reject(_arg_error("norm", "one fp32 element is required"), check)
    return _clip(grads, 0.0, norm, None, workspace, stream, check)


def clip_grads(grads, max_norm: float, norm=None, out=None, workspace=None, stream=None, check: bool = True) -> int:
    """``vlproj_clip_grads``: scales ``grads`` by ``min(1, max_norm / (norm + 1e-6))``, norm their
    global 2-norm, in place or into ``out`` (tensors of the same sizes and types, in the same
    order); ``norm`` (fp32, one element, optional) receives the norm before clipping."""
    return _clip(grads, float(max_norm), norm, grads if out is None else out, workspace, stream, check)


def clip_grads_workspace(n: int) -> int:
    """Bytes of workspace ``clip_grads`` and ``grad_norm`` need for n tensors."""
    return _size(_lib.vlproj_clip_grads_workspace(n), "vlproj_clip_grads_workspace")


def _size(n: int, what: str) -> int:
    if n < 0:
        raise VlprojError(int(n), what)
    return int(n)
