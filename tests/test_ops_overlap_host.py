"""Results that lie over an operand, a workspace or another result are refused, at
any distance of their starts and before anything is launched (no GPU needed)."""
import ctypes
import itertools
import os

import pytest

from mixture_experts_feed_amd import binding as B

BAD = B.INKLING_ERR_INVALID_ARGUMENT
BASE, STEP = 0x100000000, 0x10000000     # each buffer's own place, far from the others'


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mixture_experts_feed_amd import build
        build.build(verbose=False)
    return B.load()


def _size(fn, dims):
    n = ctypes.c_size_t(0)
    assert fn(ctypes.byref(dims), ctypes.byref(n)) == B.INKLING_OK
    return n.value


def _calls(lib):
    """name -> (buffers {name: bytes}, written names, call(addresses))"""
    R, X, E, K, N, I, H = 9000, 700, 64, 2048, 1024, 208, 1000
    g = B.GroupedDims(R, X, E, K, N, B.INKLING_BF16, B.INKLING_F32)
    gd = B.GroupedDims(R, R, E, K, N, B.INKLING_BF16, B.INKLING_BF16)
    s, n = B.SwigluDims(R, I, B.INKLING_BF16), B.NormDims(R, H, B.INKLING_NORM_LAYER, B.INKLING_F32, 1e-6)
    ws, wws = _size(lib.inkling_grouped_workspace_size, g), _size(lib.inkling_grouped_weight_grad_workspace_size, g)
    ck, nws = _size(lib.inkling_swiglu_checkpoint_size, s), _size(lib.inkling_norm_backward_workspace_size, n)
    assert ws > 0 and wws > 0
    plan = dict(index=R * 4, offsets=(E + 1) * 4)
    return {
        "grouped_linear": (dict(x=X * K * 2, w=E * N * K * 2, out=R * N * 4, ws=ws, **plan), ("out", "ws"),
                           lambda a: lib.inkling_grouped_linear(ctypes.byref(g), a["x"], a["index"], a["w"],
                                                                a["offsets"], a["out"], a["ws"], ws, None)),
        "grouped_input_grad": (dict(dout=R * N * 2, w=E * N * K * 2, dx=R * K * 2, ws=ws, offsets=(E + 1) * 4),
                               ("dx", "ws"),
                               lambda a: lib.inkling_grouped_input_grad(ctypes.byref(gd), a["dout"], a["w"],
                                                                        a["offsets"], a["dx"], a["ws"], ws, None)),
        "grouped_weight_grad": (dict(dout=R * N * 2, x=X * K * 2, dw=E * N * K * 4, ws=wws, **plan), ("dw", "ws"),
                                lambda a: lib.inkling_grouped_weight_grad(ctypes.byref(g), a["dout"], a["x"],
                                                                          a["index"], a["offsets"], a["dw"], a["ws"],
                                                                          wws, None)),
        "swiglu_forward": (dict(h=R * I * 4, gamma=R * 4, count=4, act=R * I * 2, ck=ck), ("act", "ck"),
                           lambda a: lib.inkling_swiglu_forward(ctypes.byref(s), a["h"], a["gamma"], a["count"],
                                                                a["act"], a["ck"], ck, None)),
        "swiglu_backward": (dict(dact=R * I * 2, ck=ck, gamma=R * 4, count=4, dh=R * I * 4, act=R * I * 2,
                                 dgamma=R * 4), ("dh", "act", "dgamma"),
                            lambda a: lib.inkling_swiglu_backward(ctypes.byref(s), a["dact"], a["ck"], ck, a["gamma"],
                                                                  a["count"], a["dh"], a["act"], a["dgamma"], None)),
        "norm_forward": (dict(x=R * H * 4, w=H * 4, b=H * 4, out=R * H * 4, stats=R * 8), ("out", "stats"),
                         lambda a: lib.inkling_norm_forward(ctypes.byref(n), a["x"], a["w"], a["b"], a["out"],
                                                            a["stats"], None)),
        "norm_backward": (dict(dout=R * H * 4, x=R * H * 4, w=H * 4, stats=R * 8, dx=R * H * 4, dw=H * 4, db=H * 4,
                               ws=nws), ("dx", "dw", "db", "ws"),
                          lambda a: lib.inkling_norm_backward(ctypes.byref(n), a["dout"], a["x"], a["w"], a["stats"],
                                                              a["dx"], a["dw"], a["db"], a["ws"], nws, None)),
    }


NAMES = ["grouped_linear", "grouped_input_grad", "grouped_weight_grad", "swiglu_forward", "swiglu_backward",
         "norm_forward", "norm_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_overlapping_buffers(lib, name):
    sizes, written, call = _calls(lib)[name]
    place = {b: BASE + i * STEP * 4 for i, b in enumerate(sizes)}
    assert all(n < 4 * STEP for n in sizes.values())
    for w, other in itertools.product(written, sizes):
        if w == other:
            continue
        last = (sizes[other] - 1) // 16 * 16
        for at in {0, min(16, last), sizes[other] // 2 // 16 * 16, last}:
            assert call(place | {w: place[other] + at}) == BAD, (w, other, at)
        # ... from the other side: the operand begins inside the result
        inside = (sizes[w] - 1) // 16 * 16
        assert call(place | {other: place[w] + inside}) == BAD, (w, other)
