"""Host-side argument checks of the expert-block operators' C ABI (no GPU):
every refusal returns before anything is launched."""
import ctypes
import os

import pytest
import torch

from mixture_experts_feed_amd import binding as B

P = ctypes.c_void_p
FAKE, FAKE2, FAKE3, ODD = 0x10000, 0x20000, 0x30000, 0x10008
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mixture_experts_feed_amd import build
        build.build(verbose=False)
    return B.load()


def _grouped(**kw):
    d = dict(rows=100, x_rows=100, n_groups=4, in_features=64, out_features=40, dtype=B.INKLING_BF16,
             out_dtype=B.INKLING_BF16)
    d.update(kw)
    return B.GroupedDims(d["rows"], d["x_rows"], d["n_groups"], d["in_features"], d["out_features"], d["dtype"],
                         d["out_dtype"])


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(x_rows=-1), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(n_groups=0), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(in_features=0), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(out_features=-8), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(n_groups=513), B.INKLING_ERR_UNSUPPORTED),
    (dict(in_features=60), B.INKLING_ERR_UNSUPPORTED),
    (dict(out_features=36), B.INKLING_ERR_UNSUPPORTED),
    (dict(in_features=(1 << 20) + 8), B.INKLING_ERR_UNSUPPORTED),
    (dict(dtype=2), B.INKLING_ERR_UNSUPPORTED),
    (dict(out_dtype=-1), B.INKLING_ERR_UNSUPPORTED),
    (dict(rows=2 ** 31, x_rows=2 ** 31), B.INKLING_ERR_UNSUPPORTED),
    (dict(x_rows=2 ** 31), B.INKLING_ERR_UNSUPPORTED),
])
def test_grouped_dims(lib, kw, code):
    d, n = _grouped(**kw), ctypes.c_size_t(0)
    assert lib.inkling_grouped_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert lib.inkling_grouped_weight_grad_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert lib.inkling_grouped_linear(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE2, FAKE, BIG, None) == code
    assert lib.inkling_grouped_input_grad(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE2, FAKE, BIG, None) == code
    assert lib.inkling_grouped_weight_grad(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE2, FAKE, BIG, None) == code


def test_grouped_pointers(lib):
    d = _grouped()
    bad = B.INKLING_ERR_INVALID_ARGUMENT
    fwd = lambda x=FAKE, i=None, w=FAKE2, o=FAKE, out=FAKE3, ws=FAKE, n=BIG, dd=d: lib.inkling_grouped_linear(  # noqa: E731
        ctypes.byref(dd), x, i, w, o, out, ws, n, None)
    for kw in (dict(x=None), dict(w=None), dict(o=None), dict(out=None), dict(out=FAKE), dict(out=FAKE2),
               dict(x=ODD), dict(w=ODD), dict(out=ODD), dict(o=FAKE + 2), dict(i=FAKE + 1), dict(ws=ODD)):
        assert fwd(**kw) == bad, kw
    large = _grouped(rows=9000, x_rows=9000, n_groups=64, in_features=2048, out_features=2048)
    assert fwd(dd=large, ws=None) == B.INKLING_ERR_WORKSPACE
    assert fwd(dd=large, n=64) == B.INKLING_ERR_WORKSPACE
    assert fwd(dd=_grouped(x_rows=99)) == bad                       # no row index: x has a row for each row
    assert fwd(dd=_grouped(x_rows=0), i=FAKE) == bad                # an index into nothing
    assert lib.inkling_grouped_linear(None, FAKE, None, FAKE, FAKE, FAKE2, FAKE, BIG, None) == bad
    dx = lambda d_=FAKE, w=FAKE2, o=FAKE, out=FAKE3: lib.inkling_grouped_input_grad(  # noqa: E731
        ctypes.byref(d), d_, w, o, out, FAKE, BIG, None)
    for kw in (dict(d_=None), dict(w=None), dict(o=None), dict(out=None), dict(out=FAKE2), dict(d_=ODD)):
        assert dx(**kw) == bad, kw
    dw = lambda d_=FAKE, x=FAKE2, i=None, o=FAKE, out=FAKE3, n=BIG: lib.inkling_grouped_weight_grad(  # noqa: E731
        ctypes.byref(d), d_, x, i, o, out, FAKE, n, None)
    for kw in (dict(d_=None), dict(x=None), dict(o=None), dict(out=None), dict(out=FAKE2), dict(x=ODD),
               dict(out=ODD)):
        assert dw(**kw) == bad, kw
    n = ctypes.c_size_t(0)
    big = _grouped(n_groups=64, in_features=2048, out_features=2048)
    assert lib.inkling_grouped_weight_grad_workspace_size(ctypes.byref(big), ctypes.byref(n)) == 0
    assert n.value > 0
    assert lib.inkling_grouped_weight_grad(ctypes.byref(big), FAKE, FAKE2, FAKE, FAKE, FAKE3, FAKE, n.value - 1,
                                           None) == B.INKLING_ERR_WORKSPACE
    assert lib.inkling_grouped_workspace_size(ctypes.byref(d), None) == bad


def test_grouped_tile_count_limit(lib):
    """2^31 - 257 rows against 2^20 columns are more output tiles than the kernels count."""
    d = _grouped(rows=2 ** 31 - 257, x_rows=2 ** 31 - 257, out_features=1 << 20)
    assert lib.inkling_grouped_linear(ctypes.byref(d), FAKE, None, FAKE2, FAKE, FAKE3, FAKE, 1 << 50,
                                      None) == B.INKLING_ERR_UNSUPPORTED


def test_grouped_launch_size_limit(lib):
    """fp32 products launch 256 threads for each 64 x 64 tile, and a launch has fewer than
    2^32: 2^16 row tiles (and one for the ragged end) against 2^8 column tiles are too many."""
    d = _grouped(rows=1 << 22, x_rows=1 << 22, n_groups=1, in_features=1 << 14, out_features=1 << 14,
                 dtype=B.INKLING_F32, out_dtype=B.INKLING_F32)
    un = B.INKLING_ERR_UNSUPPORTED
    assert lib.inkling_grouped_linear(ctypes.byref(d), FAKE, None, FAKE2, FAKE, FAKE3, None, 0, None) == un
    assert lib.inkling_grouped_input_grad(ctypes.byref(d), FAKE, FAKE2, FAKE, FAKE3, None, 0, None) == un
    d = _grouped(n_groups=64, in_features=1 << 15, out_features=1 << 15, dtype=B.INKLING_F32,
                 out_dtype=B.INKLING_F32)
    assert lib.inkling_grouped_weight_grad(ctypes.byref(d), FAKE, FAKE2, None, FAKE, FAKE3, None, 0, None) == un


def test_grouped_no_rows_is_a_noop(lib):
    d = _grouped(rows=0, x_rows=0)
    assert lib.inkling_grouped_linear(ctypes.byref(d), None, None, None, None, None, None, 0, None) == B.INKLING_OK
    assert lib.inkling_grouped_input_grad(ctypes.byref(d), None, None, None, None, None, 0, None) == B.INKLING_OK


def _swiglu(**kw):
    d = dict(rows=100, intermediate=64, dtype=B.INKLING_BF16) | kw
    return B.SwigluDims(d["rows"], d["intermediate"], d["dtype"])


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(intermediate=0), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(intermediate=24), B.INKLING_ERR_UNSUPPORTED),
    (dict(intermediate=(1 << 20) + 16), B.INKLING_ERR_UNSUPPORTED),
    (dict(dtype=2), B.INKLING_ERR_UNSUPPORTED),
    (dict(rows=2 ** 31), B.INKLING_ERR_UNSUPPORTED),
])
def test_swiglu_dims(lib, kw, code):
    d, n = _swiglu(**kw), ctypes.c_size_t(0)
    assert lib.inkling_swiglu_checkpoint_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert lib.inkling_swiglu_forward(ctypes.byref(d), FAKE, None, None, FAKE2, FAKE3, BIG, None) == code
    assert lib.inkling_swiglu_backward(ctypes.byref(d), FAKE, FAKE2, BIG, None, None, FAKE3, None, None, None) == code


def test_swiglu_pointers(lib):
    d, n = _swiglu(), ctypes.c_size_t(0)
    bad = B.INKLING_ERR_INVALID_ARGUMENT
    assert lib.inkling_swiglu_checkpoint_size(ctypes.byref(d), None) == bad
    assert lib.inkling_swiglu_checkpoint_size(ctypes.byref(d), ctypes.byref(n)) == 0
    assert n.value == 100 * 128 + 100 * 4
    fwd = lambda h=FAKE, g=None, c=None, act=FAKE2, ck=FAKE3, size=n.value: lib.inkling_swiglu_forward(  # noqa: E731
        ctypes.byref(d), h, g, c, act, ck, size, None)
    for kw in (dict(h=None), dict(act=None), dict(act=FAKE), dict(ck=FAKE), dict(ck=FAKE2), dict(h=ODD),
               dict(act=ODD), dict(ck=ODD), dict(g=FAKE + 2), dict(c=FAKE + 1)):
        assert fwd(**kw) == bad, kw
    assert fwd(size=n.value - 1) == B.INKLING_ERR_WORKSPACE
    bwd = lambda da=FAKE, ck=FAKE2, size=n.value, g=None, dh=FAKE3, act=None, dg=None: (  # noqa: E731
        lib.inkling_swiglu_backward(ctypes.byref(d), da, ck, size, g, None, dh, act, dg, None))
    for kw in (dict(da=None), dict(ck=None), dict(dh=None), dict(dh=FAKE), dict(dh=FAKE2), dict(act=FAKE),
               dict(act=FAKE2), dict(act=FAKE3), dict(da=ODD), dict(ck=ODD), dict(dh=ODD), dict(act=ODD),
               dict(dg=FAKE3), dict(g=0x50000, dg=0x50000), dict(dg=0x50002)):
        assert bwd(**kw) == bad, kw
    assert bwd(size=n.value - 1) == B.INKLING_ERR_WORKSPACE
    e = _swiglu(rows=0)
    assert lib.inkling_swiglu_forward(ctypes.byref(e), None, None, None, None, None, 0, None) == B.INKLING_OK
    assert lib.inkling_swiglu_backward(ctypes.byref(e), None, None, 0, None, None, None, None, None,
                                       None) == B.INKLING_OK


def _norm(**kw):
    d = dict(rows=100, hidden=64, kind=B.INKLING_NORM_LAYER, dtype=B.INKLING_BF16, eps=1e-6) | kw
    return B.NormDims(d["rows"], d["hidden"], d["kind"], d["dtype"], d["eps"])


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(hidden=0), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(eps=-1e-6), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(eps=float("nan")), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(eps=float("inf")), B.INKLING_ERR_INVALID_ARGUMENT),
    (dict(kind=2), B.INKLING_ERR_UNSUPPORTED),
    (dict(dtype=2), B.INKLING_ERR_UNSUPPORTED),
    (dict(hidden=16385), B.INKLING_ERR_UNSUPPORTED),
    (dict(rows=2 ** 31 - 65536), B.INKLING_ERR_UNSUPPORTED),
])
def test_norm_dims(lib, kw, code):
    d, n = _norm(**kw), ctypes.c_size_t(0)
    assert lib.inkling_norm_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert lib.inkling_norm_forward(ctypes.byref(d), FAKE, FAKE, None, FAKE2, None, None) == code
    assert lib.inkling_norm_backward(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE2, FAKE3, None, FAKE, BIG,
                                     None) == code


def test_norm_pointers(lib):
    d, r, n = _norm(), _norm(kind=B.INKLING_NORM_RMS), ctypes.c_size_t(0)
    bad = B.INKLING_ERR_INVALID_ARGUMENT
    fwd = lambda x=FAKE, w=FAKE3, b=None, out=FAKE2, st=None, dd=d: lib.inkling_norm_forward(  # noqa: E731
        ctypes.byref(dd), x, w, b, out, st, None)
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(out=FAKE), dict(x=ODD), dict(w=ODD), dict(b=ODD),
               dict(out=ODD), dict(st=ODD), dict(dd=r, b=FAKE)):
        assert fwd(**kw) == bad, kw
    assert lib.inkling_norm_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    bwd = lambda dy=FAKE, x=FAKE2, w=FAKE3, st=FAKE, dx=0x40000, dw=0x50000, db=None, ws=FAKE, size=n.value, dd=d: (  # noqa: E731
        lib.inkling_norm_backward(ctypes.byref(dd), dy, x, w, st, dx, dw, db, ws, size, None))
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(st=None), dict(dx=None), dict(dw=None), dict(dx=FAKE),
               dict(dx=FAKE2), dict(db=0x50000), dict(dw=FAKE3), dict(dy=ODD), dict(x=ODD), dict(dx=ODD),
               dict(dw=0x50008), dict(db=0x60008), dict(dd=r, db=0x60000), dict(ws=ODD)):
        assert bwd(**kw) == bad, kw
    assert bwd(ws=None) == B.INKLING_ERR_WORKSPACE
    assert bwd(size=n.value - 1) == B.INKLING_ERR_WORKSPACE
    assert lib.inkling_norm_forward(ctypes.byref(_norm(rows=0)), None, None, None, None, None, None) == B.INKLING_OK


def test_a_plan_holds_values_not_tensors(lib):
    """eps may come as a 0-d tensor; changing it in place must reach the next call."""
    seen = []
    real = B._call
    x, w, out = torch.zeros((2, 8)), torch.ones(8), torch.zeros((2, 8))
    eps = torch.tensor(1e-3)
    B._call = lambda dev, name, dims, *a: seen.append(ctypes.cast(dims, ctypes.POINTER(B.NormDims)).contents.eps)
    checks, operand, B._norm_checks, B._operand = B._norm_checks, B._operand, lambda *a: None, lambda *a: None
    try:
        B.norm_forward(x, w, eps=eps, out=out, save=False)
        eps.fill_(0.5)
        B.norm_forward(x, w, eps=eps, out=out, save=False)
    finally:
        B._call, B._norm_checks, B._operand = real, checks, operand
    assert seen[0] == eps.new_tensor(1e-3).item() and seen[1] == 0.5


def test_a_wanted_dtype_must_be_that_of_the_given_result():
    assert B._result_dtype("out", None, None, torch.bfloat16) is torch.bfloat16
    assert B._result_dtype("out", None, torch.float32, torch.bfloat16) is torch.float32
    t = torch.zeros(1)
    assert B._result_dtype("out", t, None, torch.bfloat16) is torch.float32
    assert B._result_dtype("out", t, torch.float32, torch.bfloat16) is torch.float32
    with pytest.raises(ValueError):
        B._result_dtype("out", t, torch.bfloat16, torch.float32)
