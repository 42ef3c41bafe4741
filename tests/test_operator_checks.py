"""Refusals of the training-step operators, on the CPU: the binding's checks of its tensors
and the library's own checks of sizes, types, alignment, workspaces and overlaps, all made
before any launch."""
import ctypes

import pytest
import torch

import vision_language_projector_b200 as vp
from vision_language_projector_b200 import operators as ops


class _Fake:
    """Stands in for a CUDA tensor on this machine: what the binding's checks look at."""

    is_cuda = True

    def __init__(self, shape, dtype=torch.float32, strides=None, device=0, ptr=0x10000000):
        self.shape, self.dtype, self._device, self._ptr = tuple(shape), dtype, device, ptr
        dense = []
        n = 1
        for d in reversed(self.shape):
            dense.insert(0, n)
            n *= max(d, 1)
        self._strides = tuple(strides) if strides else tuple(dense)
        self._dense = strides is None or self._strides == tuple(dense)

    device = property(lambda self: f"cuda:{self._device}")

    def get_device(self):
        return self._device

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def is_contiguous(self):
        return self._dense

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def data_ptr(self):
        return self._ptr


@pytest.fixture(autouse=True)
def _device_zero(monkeypatch):
    ops._use_torch()
    monkeypatch.setattr(ops, "_current_device", lambda: 0)


def _raises(fn, name):
    with pytest.raises(vp.VlprojError) as e:
        fn(True)
    assert e.value.code == vp.ERR_INVALID_ARG and name in str(e.value)
    assert fn(False) == vp.ERR_INVALID_ARG


IDS = _Fake((10,), torch.int64, ptr=0x40000000)


def test_embed_tensors():
    table, out = _Fake((7, 8)), _Fake((10, 8), ptr=0x20000000)

    def call(ids=IDS, t=table, o=out, **kw):
        return lambda check: vp.embed(ids, t, o, check=check, **kw)

    _raises(call(ids=torch.zeros(10, dtype=torch.int64)), "input_ids")       # host memory
    _raises(call(ids=_Fake((10,), torch.int32)), "input_ids")
    _raises(call(t=_Fake((7, 8), torch.float64)), "table")
    _raises(call(t=_Fake((7, 8), device=1)), "table")                        # another device
    _raises(call(t=_Fake((7, 8), strides=(16, 2))), "table")                 # elements apart
    _raises(call(t=_Fake((7, 8), strides=(4, 1))), "table")                  # rows overlap
    _raises(call(t=_Fake((7, 8), strides=(0, 1))), "table")                  # a broadcast row
    _raises(call(o=_Fake((9, 8))), "out")                                    # fewer rows than ids
    _raises(call(o=_Fake((10, 9))), "out")
    _raises(call(status=_Fake((2,), torch.int32)), "status")
    _raises(call(status=_Fake((1,), torch.int64)), "status")


def test_embed_backward_tensors():
    d_out, d_table, ws = _Fake((10, 8)), _Fake((7, 8), ptr=0x20000000), _Fake((1 << 20,), torch.uint8, ptr=0x30000000)

    def call(d=d_out, t=d_table, w=ws):
        return lambda check: vp.embed_backward(IDS, d, t, workspace=w, check=check)

    _raises(call(d=_Fake((9, 8))), "d_out")
    _raises(call(t=_Fake((7, 9))), "d_table")
    _raises(call(t=_Fake((7, 8), torch.bfloat16)), "d_table")
    _raises(call(w=_Fake((16,), torch.uint8)), "workspace")
    _raises(call(w=_Fake((1 << 20,), torch.int32)), "workspace")


def test_layernorm_tensors():
    x, y = _Fake((10, 8)), _Fake((10, 8), ptr=0x20000000)

    def call(x=x, y=y, **kw):
        return lambda check: vp.layernorm(x, y, check=check, **kw)

    _raises(call(y=_Fake((10, 9))), "y")
    _raises(call(y=_Fake((9, 8))), "y")
    _raises(call(x=_Fake(())), "x")
    _raises(call(gamma=_Fake((8,), torch.bfloat16)), "gamma")
    _raises(call(beta=_Fake((9,))), "beta")
    _raises(call(mean=_Fake((9,))), "mean")
    _raises(call(rstd=_Fake((10, 2), strides=(3, 1))), "rstd")


def test_layernorm_backward_tensors():
    x, dy, st = _Fake((10, 8)), _Fake((10, 8), ptr=0x20000000), _Fake((10,), ptr=0x30000000)

    def call(mean=st, rstd=st, dy=dy, **kw):
        return lambda check: vp.layernorm_backward(x, mean, rstd, dy, check=check, **kw)

    _raises(call(mean=None), "mean")
    _raises(call(rstd=None), "rstd")
    _raises(call(dy=_Fake((10, 9))), "d_y")
    _raises(call(d_x=_Fake((10, 8), torch.bfloat16)), "d_x")
    _raises(call(d_x=_Fake((11, 8))), "d_x")
    _raises(call(d_gamma=_Fake((7,)), workspace=_Fake((1 << 16,), torch.uint8)), "d_gamma")
    x, dy, st = _Fake((1000, 8)), _Fake((1000, 8), ptr=0x20000000), _Fake((1000,), ptr=0x30000000)
    _raises(lambda check: vp.layernorm_backward(x, st, st, dy, d_gamma=_Fake((8,)), workspace=_Fake((63,), torch.uint8),
                                                check=check), "workspace")


def test_clip_tensors():
    a, b = _Fake((4, 4)), _Fake((3,), torch.bfloat16, ptr=0x20000000)
    ws = _Fake((1 << 16,), torch.uint8, ptr=0x30000000)

    def call(g, m=1.0, **kw):
        return lambda check: vp.clip_grads(g, m, workspace=ws, stream=0, check=check, **kw)

    _raises(call([a, torch.zeros(3)]), "grads[1]")
    _raises(call({"W1": a, "W_mid": [b, _Fake((2, 2), strides=(1, 2))]}), "grads[2]")
    _raises(call([a, b], out=[a]), "out")
    _raises(call([a, b], out=[a, a]), "out[1]")
    _raises(call([a], norm=_Fake((2,))), "norm")
    _raises(lambda check: vp.grad_norm([a], None, check=check), "norm")
    for m in (-1.0, float("inf"), float("nan")):
        _raises(call([a], m), "vlproj_clip_grads")
    _raises(call([a, a]), "vlproj_clip_grads")                                  # one tensor twice
    _raises(call([a, _Fake((4,), ptr=0x10000000 + 32)]), "vlproj_clip_grads")    # inside another
    _raises(call([a], out=[_Fake((4, 4), ptr=0x10000000 + 16)]), "vlproj_clip_grads")
    _raises(call([a], norm=_Fake((1,), ptr=0x10000000 + 60)), "vlproj_clip_grads")      # the norm inside a gradient
    other = _Fake((3,), torch.bfloat16, ptr=0x10000000 + 4)                      # an output over another gradient
    _raises(call([a, b], out=[_Fake((4, 4), ptr=0x50000000), other]), "vlproj_clip_grads")


def _embed_args(**kw):
    d = dict(input_ids=0x40000000, n_ids=10, image_token_id=5, table=0x10000000, vocab=7, table_ld=8, out=0x20000000,
             out_ld=8, N=8, scale=1.0, table_type=vp.BF16, out_type=vp.BF16, status=None)
    d.update(kw)
    return ops.EmbedArgs(**d)


@pytest.mark.parametrize("kw", [dict(n_ids=-1), dict(n_ids=1 << 31), dict(vocab=-1), dict(vocab=1 << 31), dict(N=0),
                                dict(N=(1 << 20) + 1), dict(table_ld=7), dict(out_ld=1 << 60), dict(out_ld=7), dict(table=None),
                                dict(out=None), dict(input_ids=None), dict(table_type=3), dict(out_type=vp.F16),
                                dict(out_type=vp.F32), dict(table=0x10000001), dict(out=0x20000001),
                                dict(out=0x10000000 + 96), dict(out=0x40000000)])
def test_embed_library_refusals(kw):
    assert vp._lib.vlproj_embed(_embed_args(**kw), None) == vp.ERR_INVALID_ARG


def test_null_arguments():
    for name in ("embed", "embed_backward", "layernorm", "layernorm_backward", "clip_grads"):
        assert getattr(vp._lib, "vlproj_" + name)(None, None) == vp.ERR_INVALID_ARG


def _bwd_args(**kw):
    d = dict(input_ids=0x40000000, n_ids=10, image_token_id=5, d_out=0x10000000, d_out_ld=8, d_table=0x20000000,
             d_table_ld=8, vocab=7, N=8, scale=1.0, d_out_type=vp.BF16, accumulate=0, status=None,
             workspace=0x30000000, workspace_bytes=1 << 24)
    d.update(kw)
    return ops.EmbedBackwardArgs(**d)


@pytest.mark.parametrize("kw", [dict(n_ids=-1), dict(n_ids=1 << 31), dict(vocab=-1), dict(vocab=1 << 31), dict(N=0),
                                dict(d_out_ld=7), dict(d_table_ld=7), dict(d_out=None), dict(d_table=None),
                                dict(input_ids=None), dict(d_out_type=-1), dict(workspace=None),
                                dict(workspace_bytes=0), dict(workspace=0x30000008), dict(workspace=0x30000010), dict(workspace=0x10000000),
                                dict(workspace=0x20000000), dict(d_table=0x10000000), dict(d_table=0x20000002)])
def test_embed_backward_library_refusals(kw):
    assert vp._lib.vlproj_embed_backward(_bwd_args(**kw), None) == vp.ERR_INVALID_ARG


def _ln_args(**kw):
    d = dict(x=0x10000000, x_ld=8, y=0x20000000, y_ld=8, rows=10, C=8, gamma=None, beta=None, mean=None, rstd=None,
             eps=1e-5, x_type=vp.BF16, y_type=vp.BF16)
    d.update(kw)
    return ops.LayernormArgs(**d)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(C=0), dict(C=(1 << 20) + 1), dict(x_ld=7), dict(y_ld=7), dict(x_ld=1 << 60),
                                dict(x=None), dict(y=None), dict(y=0x10000000), dict(y=0x10000000 + 32),
                                dict(gamma=0x30000002), dict(mean=0x20000004), dict(mean=0x30000000, rstd=0x30000000),
                                dict(y_type=vp.F32), dict(x_type=7), dict(rows=1 << 31)])
def test_layernorm_library_refusals(kw):
    assert vp._lib.vlproj_layernorm(_ln_args(**kw), None) == vp.ERR_INVALID_ARG


def _lnb_args(**kw):
    d = dict(x=0x10000000, x_ld=8, mean=0x50000000, rstd=0x51000000, d_y=0x20000000, d_y_ld=8, gamma=None,
             d_x=0x30000000, d_x_ld=8, d_gamma=0x40000000, d_beta=0x41000000, rows=1000, C=8, x_type=vp.BF16,
             y_type=vp.BF16, workspace=0x60000000, workspace_bytes=1 << 20)
    d.update(kw)
    return ops.LayernormBackwardArgs(**d)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(C=0), dict(x_ld=7), dict(d_y_ld=7), dict(d_x_ld=7), dict(x=None),
                                dict(d_y=None), dict(mean=None), dict(rstd=None), dict(d_x=0x10000000),
                                dict(d_x=0x20000010), dict(d_gamma=0x41000000), dict(workspace=None),
                                dict(workspace_bytes=8), dict(workspace=0x60000004), dict(workspace=0x60000010), dict(workspace=0x40000000 - 256),
                                dict(y_type=vp.F16)])
def test_layernorm_backward_library_refusals(kw):
    assert vp._lib.vlproj_layernorm_backward(_lnb_args(**kw), None) == vp.ERR_INVALID_ARG


def _clip_args(n=1, grads=(0x10000000,), out=(0x20000000,), numel=(8,), types=(vp.F32,), **kw):
    keep = [(ctypes.c_void_p * len(grads))(*grads), (ctypes.c_void_p * len(out))(*out) if out else None,
            (ctypes.c_int64 * len(numel))(*numel), (ctypes.c_int32 * len(types))(*types)]
    d = dict(n=n, max_norm=1.0, norm=0x30000000, workspace=0x60000000, workspace_bytes=1 << 20)
    d.update(kw)
    a = ops.ClipGradsArgs(**d)
    a.grads, a.numel, a.type = (ctypes.cast(keep[i], ctypes.c_void_p) for i in (0, 2, 3))
    a.out = ctypes.cast(keep[1], ctypes.c_void_p) if out else None
    a._keep = keep
    return a


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=(1 << 20) + 1), dict(numel=(-1,)), dict(types=(5,)),
                                dict(grads=(0x10000002,)), dict(out=(0x20000001,)), dict(grads=(None,)),
                                dict(out=(None,)), dict(out=None, norm=None), dict(norm=0x30000001),
                                dict(numel=(1 << 20,), workspace=None), dict(numel=(1 << 20,), workspace_bytes=8),
                                dict(numel=(1 << 20,), workspace=0x60000008),
                                dict(numel=(1 << 20,), workspace=0x60000010)])
def test_clip_library_refusals(kw):
    assert vp._lib.vlproj_clip_grads(_clip_args(**kw), None) == vp.ERR_INVALID_ARG


def test_workspace_sizes():
    assert vp.embed_backward_workspace(0, 8) >= 0 and vp.layernorm_backward_workspace(1000, 8) >= 8 * 8
    assert vp.layernorm_backward_workspace(0, 8) == vp.layernorm_backward_workspace(10, 64) == 0      # few rows need none
    assert vp.clip_grads_workspace(10000) > vp.clip_grads_workspace(1)
    for fn, bad in ((vp.embed_backward_workspace, (-1, 8)), (vp.embed_backward_workspace, (1, 0)),
                    (vp.layernorm_backward_workspace, (1, (1 << 20) + 1)), (vp.clip_grads_workspace, (-1,))):
        with pytest.raises(vp.VlprojError):
            fn(*bad)


def test_empty_calls_succeed_without_a_device():
    assert vp._lib.vlproj_embed(_embed_args(n_ids=0, out=None, input_ids=None), None) == vp.OK
    assert vp._lib.vlproj_layernorm(_ln_args(rows=0, x=None, y=None), None) == vp.OK
    assert vp._lib.vlproj_embed_backward(_bwd_args(vocab=0, d_table=None), None) == vp.OK
    assert vp.clip_grads([], 1.0) == vp.OK


@pytest.mark.parametrize("kw", [dict(out=None, norm=0x10000000 + 28), dict(out=None, norm=0x10000000),          # few gradients
                                dict(out=None, norm=0x10000000 + 28, numel=(1 << 20,)),
                                dict(numel=(1 << 20,), workspace=0x10000000), dict(numel=(1 << 20,), workspace=0x20000000 + 256),
                                dict(numel=(1 << 20,), norm=0x60000000), dict(out=None, numel=(1 << 20,), norm=0x60000000),
                                dict(out=None, numel=(1 << 20,), workspace=0x10000000 + (1 << 22) - 256),
                                dict(n=2, grads=(0x10000000, 0x60000000 + 1024), numel=(1 << 20, 8), types=(vp.F32, vp.BF16), out=None)])
def test_clip_refuses_a_norm_or_workspace_over_other_arguments(kw):
    assert vp._lib.vlproj_clip_grads(_clip_args(**kw), None) == vp.ERR_INVALID_ARG


@pytest.mark.parametrize("at", [0x20000000 + 4, 0x10000000 + 8, 0x40000000 + 8, 0x30000000 + 4, 0x70000001])
def test_status_misplaced(at):
    """The status word inside a matrix, the ids or the workspace, or not on 4 bytes."""
    if at < 0x30000000 or at >= 0x40000000:
        assert vp._lib.vlproj_embed(_embed_args(status=at), None) == vp.ERR_INVALID_ARG
    assert vp._lib.vlproj_embed_backward(_bwd_args(status=at), None) == vp.ERR_INVALID_ARG


def test_misaligned_ids():
    for at in (0x40000004, 0x40000001):
        assert vp._lib.vlproj_embed(_embed_args(input_ids=at), None) == vp.ERR_INVALID_ARG
        assert vp._lib.vlproj_embed_backward(_bwd_args(input_ids=at), None) == vp.ERR_INVALID_ARG


@pytest.mark.parametrize("token", [1 << 63, (1 << 64) + 5, -(1 << 63) - 1])
def test_token_ids_beyond_int64(token):
    table, out = _Fake((7, 8)), _Fake((10, 8), ptr=0x20000000)
    # an empty list of ids: the library accepts the call without a device
    none = _Fake((0,), torch.int64, ptr=0)
    assert vp.embed(none, table, out, image_token_id=(1 << 63) - 1, stream=0) == vp.OK
    _raises(lambda check: vp.embed(none, table, out, image_token_id=token, stream=0, check=check), "image_token_id")
    ws = _Fake((1 << 20,), torch.uint8, ptr=0x30000000)
    _raises(lambda check: vp.embed_backward(IDS, out, _Fake((0, 8), ptr=0), image_token_id=token, workspace=ws, stream=0,
                                            check=check), "image_token_id")
