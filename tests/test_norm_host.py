"""Refusals of the gradient-norm and clipping calls (no GPU call is made)."""
import ctypes
import math

import pytest
import torch

import fsdp_sharded_state_amd as fs

GOOD = 1 << 20     # addresses that are never read: every call here is refused before it launches
TOTAL, NORM, WS = 1 << 30, (1 << 30) + 64, 1 << 31


def _list(ptrs, numels, codes):
    n = len(ptrs)
    return (ctypes.c_void_p * max(1, n))(*ptrs), (ctypes.c_int64 * max(1, n))(*numels), (ctypes.c_int32 * max(1, n))(*codes)


def _norm(ptrs=(GOOD,), numels=(100,), codes=(1,), n=None, kind=1, total=TOTAL, norm=NORM, ws=WS, nbytes=1 << 24):
    p, m, c = _list(ptrs, numels, codes)
    return fs.lib().fs_grad_norm(len(ptrs) if n is None else n, p, m, c, kind, 0, total, norm, ws, nbytes, None)


def _clip(ptrs=(GOOD,), numels=(100,), codes=(1,), n=None, kind=1, total=TOTAL, norm=NORM, max_norm=1.0, eps=1e-6,
          clip=True):
    p, m, c = _list(ptrs, numels, codes)
    cl = fs.Clip(total, max_norm, eps, kind)
    return fs.lib().fs_clip_grads(len(ptrs) if n is None else n, p, m, c, ctypes.byref(cl) if clip else None, norm, None)


LIST_REFUSALS = [
    (dict(n=-1), fs.FS_E_INVAL),
    (dict(numels=(-1,)), fs.FS_E_INVAL),
    (dict(codes=(2,)), fs.FS_E_DTYPE),
    (dict(ptrs=(None,)), fs.FS_E_INVAL),
    (dict(ptrs=(GOOD + 2,)), fs.FS_E_ALIGN),
    (dict(ptrs=(GOOD + 1,), codes=(0,)), fs.FS_E_ALIGN),
    (dict(numels=(1 << 61,)), fs.FS_E_OVERFLOW),
    (dict(numels=(1 << 52,)), fs.FS_E_OVERFLOW),            # more tiles than a grid holds
    (dict(kind=0), fs.FS_E_UNSUPPORTED),
    (dict(kind=3), fs.FS_E_UNSUPPORTED),
    (dict(total=None), fs.FS_E_INVAL),
    (dict(total=TOTAL + 4), fs.FS_E_ALIGN),
    (dict(norm=NORM + 2), fs.FS_E_ALIGN),
    (dict(norm=TOTAL + 4), fs.FS_E_INVAL),                  # inside the total
    (dict(ptrs=(TOTAL - 40,)), fs.FS_E_INVAL),              # the total lies inside the tensor
    (dict(ptrs=(NORM - 48,), numels=(13,)), fs.FS_E_INVAL),  # the norm is its last element
]


@pytest.mark.parametrize("kw,code", LIST_REFUSALS)
def test_list_refusals(kw, code):
    assert _norm(**kw) == code and fs.lib().fs_last_error().startswith(b"fs_grad_norm")
    assert _clip(**kw) == code and fs.lib().fs_last_error().startswith(b"fs_clip_grads")


@pytest.mark.parametrize("call", [_norm, _clip])
def test_a_tensor_beyond_one_launch_is_refused(call):
    """More than 2^32 threads' worth of one tensor; a list of that many bytes is cut."""
    assert call(ptrs=(1 << 44,), numels=(1 << 36,)) == fs.FS_E_OVERFLOW
    assert b"tensor 0" in fs.lib().fs_last_error()
    assert call(ptrs=(1 << 44,), numels=(1 << 37,), codes=(0,)) == fs.FS_E_OVERFLOW
    need = ctypes.c_int64()
    m, c = (ctypes.c_int64 * 2)(1 << 36, 1), (ctypes.c_int32 * 2)(1, 1)
    assert fs.lib().fs_grad_norm_workspace(2, m, c, ctypes.byref(need)) == fs.FS_E_OVERFLOW
    m = (ctypes.c_int64 * 2)(1 << 34, 1 << 34)
    assert fs.lib().fs_grad_norm_workspace(2, m, c, ctypes.byref(need)) == 0
    assert need.value >= 8 * (1 << 24)     # 8 KB of gradients to a partial total


def test_a_bad_tensor_is_named():
    assert _norm(ptrs=(GOOD, GOOD + 4096, GOOD + 8194), numels=(1, 2, 3), codes=(0, 1, 1)) == fs.FS_E_ALIGN
    assert b"tensor 2" in fs.lib().fs_last_error()


def test_workspace_refusals():
    need = ctypes.c_int64()
    m, c = (ctypes.c_int64 * 1)(1 << 24), (ctypes.c_int32 * 1)(1)
    L = fs.lib()
    assert L.fs_grad_norm_workspace(1, m, c, ctypes.byref(need)) == 0 and need.value > 0
    big = dict(numels=(1 << 24,), ptrs=(1 << 34,))
    assert _norm(ws=None, **big) == fs.FS_E_INVAL
    assert _norm(ws=WS + 4, **big) == fs.FS_E_ALIGN
    assert _norm(nbytes=need.value - 1, **big) == fs.FS_E_INVAL
    assert _norm(ws=TOTAL, **big) == fs.FS_E_INVAL
    assert _norm(ws=(1 << 34) + 4096, **big) == fs.FS_E_INVAL
    assert L.fs_grad_norm_workspace(1, m, c, None) == fs.FS_E_INVAL
    assert L.fs_grad_norm_workspace(-1, m, c, ctypes.byref(need)) == fs.FS_E_INVAL
    assert L.fs_grad_norm_workspace(0, None, None, ctypes.byref(need)) == 0 and need.value == 0
    assert L.fs_reduce_shard_norm_workspace(-1, ctypes.byref(need)) == fs.FS_E_INVAL
    assert L.fs_reduce_shard_norm_workspace(1, None) == fs.FS_E_INVAL


@pytest.mark.parametrize("kw,code", [
    (dict(clip=False), fs.FS_E_INVAL),
    (dict(max_norm=-1.0), fs.FS_E_INVAL),
    (dict(max_norm=math.nan), fs.FS_E_INVAL),
    (dict(eps=-1e-9), fs.FS_E_INVAL),
    (dict(eps=math.nan), fs.FS_E_INVAL),
    (dict(eps=math.inf), fs.FS_E_INVAL),
    (dict(ptrs=(GOOD, GOOD), numels=(4, 4), codes=(1, 1)), fs.FS_E_INVAL),                    # the same tensor twice
    (dict(ptrs=(GOOD + 4096, GOOD, GOOD + 8192), numels=(8, 1025, 8), codes=(1, 1, 1)), fs.FS_E_INVAL),
    (dict(ptrs=(GOOD + 2, GOOD), numels=(8, 2), codes=(0, 0)), fs.FS_E_INVAL),                # half an fp32 apart
])
def test_clip_refusals(kw, code):
    assert _clip(**kw) == code


def _reduce(n=64, world=2, acc=1, dt=1, slices=(GOOD, GOOD + 4096), out=1 << 24, kind=1, total=TOTAL, norm=NORM,
            ws=WS, nbytes=1 << 24):
    arr = (ctypes.c_void_p * max(1, len(slices)))(*slices)
    return fs.lib().fs_reduce_shard_norm(n, world, acc, dt, arr, out, kind, 0, total, norm, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), fs.FS_E_INVAL),
    (dict(world=0), fs.FS_E_INVAL),
    (dict(dt=5), fs.FS_E_DTYPE),
    (dict(world=40, dt=0, slices=(GOOD,) * 40), fs.FS_E_UNSUPPORTED),
    (dict(slices=(GOOD, None)), fs.FS_E_INVAL),
    (dict(slices=(GOOD, GOOD + 1)), fs.FS_E_ALIGN),
    (dict(out=GOOD), fs.FS_E_INVAL),                 # out overlaps a slice
    (dict(out=None), fs.FS_E_INVAL),
    (dict(kind=7), fs.FS_E_UNSUPPORTED),
    (dict(total=None), fs.FS_E_INVAL),
    (dict(total=TOTAL + 1), fs.FS_E_ALIGN),
    (dict(total=GOOD + 8), fs.FS_E_INVAL),           # inside a slice
    (dict(total=(1 << 24) + 8), fs.FS_E_INVAL),      # inside out
    (dict(norm=(1 << 24) + 8), fs.FS_E_INVAL),
    (dict(norm=GOOD + 4096), fs.FS_E_INVAL),
    (dict(n=1 << 20, slices=(1 << 34, 1 << 35), ws=None), fs.FS_E_INVAL),
    (dict(n=1 << 20, slices=(1 << 34, 1 << 35), nbytes=8), fs.FS_E_INVAL),
    (dict(n=1 << 20, slices=(1 << 34, 1 << 35), ws=WS + 4), fs.FS_E_ALIGN),
    (dict(n=1 << 20, slices=(1 << 34, 1 << 35), ws=(1 << 24) + 64), fs.FS_E_INVAL),   # inside out
    (dict(n=1 << 20, slices=(1 << 34, 1 << 35), ws=(1 << 34) + 64), fs.FS_E_INVAL),   # inside a slice
])
def test_reduce_norm_refusals(kw, code):
    assert _reduce(**kw) == code and fs.lib().fs_last_error().startswith(b"fs_reduce_shard_norm")


def _adamw(n=64, th=1 << 20, m=1 << 21, v=1 << 22, g=1 << 23, gd=1, p=1 << 24, total=TOTAL, max_norm=1.0, eps=1e-6,
           kind=1, clip=True, step=1):
    hp = fs.AdamWHparams(1e-3, 0.9, 0.999, 1e-8, 0.01, 0, step)
    cl = fs.Clip(total, max_norm, eps, kind)
    return fs.lib().fs_adamw_step_clip(n, th, m, v, g, gd, p, ctypes.byref(hp), ctypes.byref(cl) if clip else None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(clip=False), fs.FS_E_INVAL),
    (dict(total=None), fs.FS_E_INVAL),
    (dict(total=TOTAL + 4), fs.FS_E_ALIGN),
    (dict(kind=0), fs.FS_E_UNSUPPORTED),
    (dict(max_norm=-0.5), fs.FS_E_INVAL),
    (dict(eps=math.nan), fs.FS_E_INVAL),
    (dict(total=1 << 20), fs.FS_E_INVAL),            # inside master
    (dict(total=(1 << 23) + 8), fs.FS_E_INVAL),      # inside the gradient
    (dict(n=-1), fs.FS_E_INVAL),
    (dict(step=0), fs.FS_E_INVAL),
    (dict(gd=4), fs.FS_E_DTYPE),
    (dict(m=1 << 20), fs.FS_E_INVAL),
    (dict(v=(1 << 22) + 2), fs.FS_E_ALIGN),
])
def test_adamw_clip_refusals(kw, code):
    assert _adamw(**kw) == code and fs.lib().fs_last_error().startswith(b"fs_adamw_step_clip")


def test_binding_refusals():
    t = torch.zeros(8)
    total, norm = torch.zeros(1, dtype=torch.float64), torch.zeros(1)
    with pytest.raises(ValueError, match="GPU tensor"):
        fs.fs_grad_list([t])
    with pytest.raises(ValueError, match="GPU tensor"):
        fs.fs_grad_norm([t], total)
    with pytest.raises(ValueError, match="GPU tensor"):
        fs.fs_grad_norm([], total)
    with pytest.raises(ValueError, match="norm_type"):
        fs.fs_grad_norm([], total, norm_type=1)
    with pytest.raises(ValueError, match="float64"):
        fs.fs_clip_grads([], norm, 1.0)
    with pytest.raises(ValueError, match="float64"):
        fs.fs_clip_grads([], torch.zeros(2, dtype=torch.float64), 1.0)
    with pytest.raises(ValueError, match="slices"):
        fs.fs_reduce_shard_norm([t], t, total, world=2)
    with pytest.raises(ValueError, match="float32"):
        fs.fs_reduce_shard_norm([t, t], t.to(torch.bfloat16), total, world=2)
    with pytest.raises(ValueError, match="exp_avg must be"):
        fs.fs_adamw_step_clip(t, t[:4], t, t, total=total, max_norm=1.0)
    with pytest.raises(ValueError, match="grad must be"):
        fs.fs_adamw_step_clip(t, t, t, t.to(torch.float16), total=total, max_norm=1.0)
    with pytest.raises(ValueError, match="float64"):
        fs.fs_adamw_step_clip(t, t, t, t, total=norm, max_norm=1.0)
