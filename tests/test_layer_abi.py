"""The layer operators' argument checks: every refusal of include/da.h, with its documented code and
before any launch (fake pointers, no GPU needed), and the binding's own checks."""
import ctypes

import pytest
import torch

import block_sparse_cluster_b200 as da

OK_CODE, INVALID, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5, 9
# fake bases a terabyte apart: nothing overlaps unless a test says so
X, R, W, S, O, C, P, WS = (0x10000000000 * i for i in range(1, 9))


def _norm(rows=10, width=64, dtype=0, x=X, xs=64, r=R, rs=64, w=W, eps=1e-6, s=S, ss=64, o=O, os_=64):
    return da._lib.da_rms_norm(rows, width, dtype, x, xs, r, rs, w, eps, s, ss, o, os_, None)


def _norm_i8(rows=10, width=64, dtype=0, x=X, xs=64, r=R, rs=64, w=W, eps=1e-6, s=S, ss=64, o=O, os_=64, c=C):
    return da._lib.da_rms_norm_i8(rows, width, dtype, x, xs, r, rs, w, eps, s, ss, o, os_, c, None)


@pytest.mark.parametrize("call", [_norm, _norm_i8])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INVALID), (dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(x=None), INVALID),
    (dict(o=None), INVALID), (dict(r=None), INVALID),            # a sum without a residual
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(width=16385, xs=16385, rs=16385, ss=16385, os_=16385), UNSUPPORTED),
    (dict(rows=1 << 31), SHAPE), (dict(rows=(1 << 31) - 65535), SHAPE), (dict(rows=(1 << 31) - 65536, os_=1 << 40), SHAPE),
    (dict(rows=(1 << 24) + 1, xs=1 << 40), SHAPE), (dict(xs=-64), SHAPE), (dict(xs=1 << 41), SHAPE), (dict(os_=63), SHAPE),
    (dict(os_=0), SHAPE), (dict(ss=63), SHAPE),
    (dict(x=X + 1), ALIGN), (dict(r=R + 1), ALIGN), (dict(w=W + 1), ALIGN), (dict(s=S + 1), ALIGN),
    (dict(s=O), INVALID), (dict(o=W), INVALID), (dict(s=W), INVALID), (dict(s=X + 2), INVALID), (dict(s=R + 128), INVALID),
    (dict(s=X, ss=65), INVALID),                                 # the same base with other strides
])
def test_norm_refuses(call, kw, code):
    assert call(**kw) == code


def test_norm_forms_refuse_their_own():
    assert _norm(o=X + 2) == INVALID and _norm(o=R, os_=72) == INVALID
    assert _norm_i8(c=None) == INVALID and _norm_i8(c=C + 2) == ALIGN
    for other in ("x", "r", "w", "s"):
        assert _norm_i8(**{other: C}) == INVALID and _norm_i8(**{other: O}) == INVALID
    assert _norm_i8(o=C) == INVALID


def _quant(B=2, H=3, N=10, d=64, dtype=0, x=X, st=(1920, 640, 64), q=O, qs=192, c=C):
    strides = da._HeadStrides(*st) if st is not None else None
    return da._lib.da_quantize_i8(B, H, N, d, dtype, x, ctypes.byref(strides) if st is not None else None, q, qs, c, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=-1), INVALID), (dict(N=0), INVALID), (dict(d=0), INVALID), (dict(x=None), INVALID),
    (dict(st=None), INVALID), (dict(q=None), INVALID), (dict(c=None), INVALID), (dict(dtype=7), DTYPE),
    (dict(H=300, d=64), UNSUPPORTED), (dict(B=1 << 16, N=1 << 16), SHAPE), (dict(st=(1920, 640, -1)), SHAPE),
    (dict(qs=191), SHAPE), (dict(x=X + 1), ALIGN), (dict(c=C + 1), ALIGN), (dict(q=X), INVALID), (dict(c=X), INVALID),
    (dict(c=O), INVALID),
])
def test_quantize_refuses(kw, code):
    assert _quant(**kw) == code


def _linear(B=2, N=10, H=3, d=64, K=256, x=X, xs=256, sx=S, w=W, wstr=256, sw=R, bias=P, dtype=0, o=O,
            st=(1920, 640, 64), ws=WS, wsb=256):
    strides = da._HeadStrides(*st) if st is not None else None
    return da._lib.da_linear_i8(B, N, H, d, K, x, xs, sx, w, wstr, sw, bias, dtype, o,
                                ctypes.byref(strides) if st is not None else None, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID), (dict(K=0), INVALID),
    (dict(x=None), INVALID), (dict(sx=None), INVALID), (dict(w=None), INVALID), (dict(sw=None), INVALID),
    (dict(o=None), INVALID), (dict(st=None), INVALID), (dict(ws=None), INVALID), (dict(dtype=2), DTYPE),
    (dict(K=131072, xs=131072, wstr=131072), UNSUPPORTED), (dict(B=1 << 16, N=1 << 16), SHAPE),
    (dict(H=1 << 16, d=64), SHAPE), (dict(xs=-1), SHAPE), (dict(st=(1920, 639, 64)), SHAPE), (dict(st=(0, 640, 64)), SHAPE),
    (dict(sx=S + 2), ALIGN), (dict(sw=R + 1), ALIGN), (dict(bias=P + 3), ALIGN), (dict(o=O + 1), ALIGN),
    (dict(ws=WS + 4), ALIGN), (dict(wsb=255), WORKSPACE),
    (dict(o=X), INVALID), (dict(o=W), INVALID), (dict(o=S), INVALID), (dict(o=R), INVALID), (dict(o=P), INVALID),
    (dict(o=WS), INVALID),
])
def test_linear_refuses(kw, code):
    assert _linear(**kw) == code


def _rope(plan=True, axes=(24, 20, 20), grid=(2, 2, 4), theta=1e4, pairing=0, B=2, H=3, N=16, d=64, dtype=0, x=X,
          xs=(6144, 64, 384), pos=None, pb=0, w=None, ww=0, eps=1e-6, o=O, os_=(6144, 1024, 64)):
    p = da._RopePlan(*axes, *grid, theta, pairing)
    a = ctypes.byref(da._HeadStrides(*xs)) if xs is not None else None
    b = ctypes.byref(da._HeadStrides(*os_)) if os_ is not None else None
    return da._lib.da_rope(ctypes.byref(p) if plan else None, B, H, N, d, dtype, x, a, pos, pb, w, ww, eps, o, b, None)


@pytest.mark.parametrize("kw,code", [
    (dict(plan=False), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(N=0), INVALID), (dict(d=0), INVALID),
    (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(o=None), INVALID), (dict(os_=None), INVALID),
    (dict(dtype=2), DTYPE), (dict(d=96, axes=(32, 32, 32)), UNSUPPORTED), (dict(pairing=2), INVALID), (dict(pairing=-1), INVALID),
    (dict(theta=0.0), INVALID), (dict(theta=-1.0), INVALID), (dict(theta=0.5), INVALID), (dict(theta=float("nan")), INVALID),
    (dict(theta=float("inf")), INVALID),
    (dict(axes=(24, 21, 19)), SHAPE), (dict(axes=(24, 20, 18)), SHAPE), (dict(axes=(-2, 46, 20)), SHAPE),
    (dict(grid=(0, 2, 4)), SHAPE), (dict(grid=(1 << 16, 1 << 15, 1)), SHAPE), (dict(B=1 << 16, N=1 << 16), SHAPE),
    (dict(w=W, ww=65), SHAPE), (dict(w=W, ww=0), SHAPE), (dict(w=W, ww=64, eps=-1.0), INVALID),
    (dict(H=300, w=W, ww=300 * 64, os_=(1 << 20, 1024, 64)), UNSUPPORTED),
    (dict(os_=(6144, 1024, 56)), SHAPE), (dict(os_=(6144, 0, 64)), SHAPE), (dict(pos=P, pb=47), SHAPE), (dict(pos=P, pb=-48), SHAPE),
    (dict(x=X + 8), ALIGN), (dict(o=O + 8), ALIGN), (dict(xs=(6144, 64, 388)), ALIGN), (dict(os_=(6144, 1028, 64)), ALIGN),
    (dict(w=W + 8, ww=64), ALIGN), (dict(pos=P + 2), ALIGN),
    (dict(o=X), INVALID), (dict(o=X + 128, os_=(6144, 64, 384)), INVALID), (dict(w=O, ww=64), INVALID), (dict(pos=O), INVALID),
])
def test_rope_refuses(kw, code):
    assert _rope(**kw) == code


def test_binding_refuses_before_the_library():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    # tensors of the host are no CUDA tensors
    for f in (lambda: da.da_rms_norm(x, None, x), lambda: da.da_rms_norm_i8(x, None, q, s),
              lambda: da.da_quantize_i8(x, q, s), lambda: da.da_linear_i8(q, s, q, s, x[:, :4], q),
              lambda: da.da_rope(x.view(1, 1, 4, 64), x.view(1, 1, 4, 64), da.Rope((32, 16, 16), (1, 2, 2)))):
        with pytest.raises(da.DAError) as e:
            f()
        assert e.value.code == INVALID
    h = x.view(1, 1, 4, 64)
    for rope, word in ((da.Rope((32, 16, 16), pairing="other"), "pairing"), (da.Rope((32, 32)), "axes"),
                       (da.Rope((32, 16, 16), (1, 2)), "grid"), (da.Rope((32, 16, 1 << 40)), "axes"), ((1, 2), "Rope")):
        with pytest.raises(da.DAError, match=word) as e:
            da.da_rope(h, h, rope)
        assert e.value.code == INVALID
    for bad in (lambda: da.da_rms_norm(1, None, x), lambda: da.da_quantize_i8(x, None, s), lambda: da.da_rope(h, [], da.Rope((32, 16, 16)))):
        with pytest.raises(da.DAError) as e:
            bad()
        assert e.value.code == INVALID


def test_package_fails_loudly_without_the_marshalling_module(tmp_path):
    import os
    import shutil
    import subprocess
    import sys
    src = os.path.dirname(da.LIB_PATH)
    pkg = tmp_path / "block_sparse_cluster_b200"
    pkg.mkdir()
    for name in ("__init__.py", "layer.py", "libda.so"):
        shutil.copy(os.path.join(src, name), pkg / name)
    r = subprocess.run([sys.executable, "-c", "import block_sparse_cluster_b200"], cwd=tmp_path,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)}, capture_output=True, text=True, timeout=300)
    assert r.returncode != 0 and "ImportError" in r.stderr and "_layer_call.so is not built" in r.stderr
