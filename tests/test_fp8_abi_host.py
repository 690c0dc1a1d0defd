"""Host-side argument checks of the 8-bit floating point operators (no GPU): every
refusal returns before anything is launched."""
import ctypes
import itertools
import os

import pytest
import torch

from mixture_experts_feed_amd import binding as B

BAD, UN = B.INKLING_ERR_INVALID_ARGUMENT, B.INKLING_ERR_UNSUPPORTED
FAKE = [0x100000000 * (i + 1) for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mixture_experts_feed_amd import build
        build.build(verbose=False)
    return B.load()


def _fp8(**kw):
    d = dict(rows=100, x_rows=100, n_groups=4, in_features=256, out_features=144, out_dtype=B.INKLING_BF16) | kw
    return B.Fp8Dims(*[d[n] for n, _ in B.Fp8Dims._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(n_groups=0), BAD), (dict(in_features=0), BAD), (dict(out_features=-16), BAD), (dict(n_groups=513), UN),
    (dict(in_features=24), UN), (dict(out_features=8), UN), (dict(in_features=(1 << 20) + 16), UN),
    (dict(out_dtype=2), UN), (dict(out_dtype=-1), UN),
])
def test_dims(lib, kw, code):
    d = ctypes.byref(_fp8(**kw))
    assert lib.inkling_fp8_grouped_linear(d, FAKE[0], FAKE[1], None, FAKE[2], FAKE[3], FAKE[4], FAKE[5], None) == code
    assert lib.inkling_fp8_grouped_input_grad(d, *FAKE[:6], None) == code
    assert lib.inkling_fp8_quantize_weight(d, *FAKE[:3], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(x_rows=-1), BAD), (dict(rows=2 ** 31, x_rows=2 ** 31), UN), (dict(x_rows=2 ** 31), UN),
    # 2^31 - 257 rows against 2^20 columns: more tiles than 31 bits count
    (dict(rows=2 ** 31 - 257, x_rows=2 ** 31 - 257, in_features=1 << 20, out_features=1 << 20), UN),
    (dict(n_groups=512, out_features=1 << 20), UN),
])
def test_product_sizes(lib, kw, code):
    d = ctypes.byref(_fp8(**kw))
    assert lib.inkling_fp8_grouped_linear(d, FAKE[0], FAKE[1], None, FAKE[2], FAKE[3], FAKE[4], FAKE[5], None) == code
    assert lib.inkling_fp8_grouped_input_grad(d, *FAKE[:6], None) == code


R, E, N, K = 100, 4, 144, 256
SIZES = {
    "inkling_fp8_grouped_linear": (dict(x=R * K, x_scales=R * 8, index=R * 4, weight=E * N * K, weight_scales=E * 16,
                                        offsets=20, out=R * N * 2), ("index",)),
    "inkling_fp8_grouped_input_grad": (dict(dout=R * N, dout_scales=R * 8, weight=E * N * K, weight_scales=E * 16,
                                            offsets=20, dx=R * K * 2), ()),
    "inkling_fp8_quantize_weight": (dict(weight=E * N * K * 2, values=E * N * K, scales=E * 16), ()),
}
WRITTEN = {"inkling_fp8_grouped_linear": ("out",), "inkling_fp8_grouped_input_grad": ("dx",),
           "inkling_fp8_quantize_weight": ("values", "scales"), "inkling_fp8_quantize_rows": ("values", "scales")}


def _pointers(call, sizes, written, optional):
    at = dict(zip(sizes, FAKE))
    for n in sizes:
        if n not in optional:
            assert call(at | {n: None}) == BAD, n
        assert call(at | {n: at[n] + 2}) == BAD, n
        if n in ("x", "dout", "weight", "values", "out", "dx"):
            assert call(at | {n: at[n] + 8}) == BAD, n
    for w, other in itertools.product(written, sizes):
        if w != other:
            for off in {0, sizes[other] // 32 * 16, (sizes[other] - 1) // 16 * 16}:
                assert call(at | {w: at[other] + off}) == BAD, (w, other, off)
            assert call(at | {other: at[w] + (sizes[w] - 1) // 16 * 16}) == BAD, (w, other)


@pytest.mark.parametrize("name", SIZES)
def test_pointers(lib, name):
    sizes, optional = SIZES[name]
    d = _fp8()
    _pointers(lambda a: getattr(lib, name)(ctypes.byref(d), *a.values(), None), sizes, WRITTEN[name], optional)
    assert getattr(lib, name)(None, *FAKE[:len(sizes)], None) == BAD


def test_product_calls(lib):
    call = lambda d, index=None, offsets=FAKE[5]: lib.inkling_fp8_grouped_linear(  # noqa: E731
        ctypes.byref(d), FAKE[0], FAKE[1], index, FAKE[3], FAKE[4], offsets, FAKE[6], None)
    assert call(_fp8(x_rows=99)) == BAD                    # no row index: x has a row for each row
    assert call(_fp8(x_rows=0), index=FAKE[2]) == BAD      # an index into nothing
    assert call(_fp8(), offsets=None) == BAD               # several groups need offsets
    none = [None] * 7
    assert lib.inkling_fp8_grouped_linear(ctypes.byref(_fp8(rows=0, x_rows=0)), *none, None) == B.INKLING_OK
    assert lib.inkling_fp8_grouped_input_grad(ctypes.byref(_fp8(rows=0)), *none[:6], None) == B.INKLING_OK


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(cols=40), UN), (dict(cols=(1 << 20) + 16), UN), (dict(dtype=2), UN),
    (dict(rows=2 ** 31), UN), (dict(rows=2 ** 30, cols=384), UN),
])
def test_quantize_rows_dims(lib, kw, code):
    d = dict(rows=10, cols=64, dtype=B.INKLING_F32) | kw
    dims = B.QuantDims(d["rows"], d["cols"], d["dtype"])
    assert lib.inkling_fp8_quantize_rows(ctypes.byref(dims), FAKE[0], None, FAKE[1], FAKE[2], None) == code


def test_quantize_rows_pointers(lib):
    d = B.QuantDims(100, 272, B.INKLING_F32)
    _pointers(lambda a: lib.inkling_fp8_quantize_rows(ctypes.byref(d), a["x"], a["count"], a["values"], a["scales"], None),
              dict(x=100 * 272 * 4, count=4, values=100 * 272, scales=1200), WRITTEN["inkling_fp8_quantize_rows"],
              ("count",))
    none = B.QuantDims(0, 272, B.INKLING_F32)
    assert lib.inkling_fp8_quantize_rows(ctypes.byref(none), None, None, None, None, None) == B.INKLING_OK
    assert lib.inkling_fp8_quantize_rows(None, *FAKE[:4], None) == BAD


def test_sizes_past_32_bits_are_value_errors():
    bf = torch.bfloat16
    for make in (lambda v: B.make_quant_dims(1, v, bf), lambda v: B._quant_plan(1, v, bf),
                 lambda v: B.make_fp8_dims(1, 1, v, 16, 16, bf), lambda v: B.make_fp8_dims(1, 1, 1, v, 16, bf),
                 lambda v: B._fp8_plan(1, 1, 1, 16, v, bf)):
        for v in (2 ** 31, 2 ** 32 + 64, -2 ** 32 + 64):
            with pytest.raises(ValueError):
                make(v)
