"""Host-side argument checks of the operators that sort tokens by expert and back
(no GPU): every refusal returns before anything is launched."""
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


def _order(**kw):
    d = dict(T=100, n_routed=8, top_k=2) | kw
    return B.OrderDims(d["T"], d["n_routed"], d["top_k"])


def _dispatch(**kw):
    d = dict(T=100, rows=200, top_k=2, hidden=64, token_dtype=B.INKLING_BF16, rows_dtype=B.INKLING_F32) | kw
    return B.DispatchDims(*[d[n] for n, _ in B.DispatchDims._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(n_routed=0), BAD), (dict(top_k=0), BAD), (dict(n_routed=513), UN), (dict(top_k=33), UN),
    (dict(T=2 ** 30), UN), (dict(T=2 ** 31, top_k=1), UN), (dict(T=2 ** 60, top_k=32), UN),
])
def test_order_dims(lib, kw, code):
    d, n = _order(**kw), ctypes.c_size_t(0)
    assert lib.inkling_expert_order_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert lib.inkling_expert_order(ctypes.byref(d), *FAKE[:7], 1 << 40, None) == code


def _order_call(lib, d, at, size=1 << 40):
    return lib.inkling_expert_order(ctypes.byref(d), *[at[n] for n in ("topk", "mask", "counts", "offsets", "slots",
                                                                       "positions", "ws")], size, None)


def test_order_pointers(lib):
    d = _order(T=9000)
    at = dict(zip(("topk", "mask", "counts", "offsets", "slots", "positions", "ws"), FAKE))
    n = ctypes.c_size_t(0)
    assert lib.inkling_expert_order_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.inkling_expert_order_workspace_size(ctypes.byref(d), None) == BAD
    assert lib.inkling_expert_order_workspace_size(None, ctypes.byref(n)) == BAD
    for name in ("topk", "offsets", "positions"):
        assert _order_call(lib, d, at | {name: None}) == BAD, name
    for name in ("topk", "counts", "offsets", "slots", "positions"):
        assert _order_call(lib, d, at | {name: at[name] + 2}) == BAD, name
    assert _order_call(lib, d, at | {"ws": at["ws"] + 8}) == BAD
    assert _order_call(lib, d, at | {"ws": None}) == B.INKLING_ERR_WORKSPACE
    assert _order_call(lib, d, at, n.value - 1) == B.INKLING_ERR_WORKSPACE
    sizes = dict(topk=72000, mask=9000, counts=32, offsets=36, slots=72000, positions=72000, ws=n.value)
    for w, other in itertools.product(("counts", "offsets", "slots", "positions", "ws"), sizes):
        if w != other:
            last = (sizes[other] - 1) // 16 * 16
            for off in {0, sizes[other] // 32 * 16, last}:
                assert _order_call(lib, d, at | {w: at[other] + off}) == BAD, (w, other, off)
    small = _order(T=10)
    assert lib.inkling_expert_order_workspace_size(ctypes.byref(small), ctypes.byref(n)) == 0 and n.value == 0


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(rows=-1), BAD), (dict(top_k=0), BAD), (dict(hidden=0), BAD), (dict(top_k=33), UN),
    (dict(hidden=(1 << 20) + 1), UN), (dict(token_dtype=2), UN), (dict(rows_dtype=-1), UN), (dict(rows=2 ** 31), UN),
    (dict(T=2 ** 30), UN), (dict(T=1 << 25, top_k=1), UN), (dict(T=1 << 20, hidden=8192), UN), (dict(T=2 ** 61), UN),
])
def test_row_dims(lib, kw, code):
    d = ctypes.byref(_dispatch(**kw))
    f = FAKE
    assert lib.inkling_dispatch_forward(d, *f[:4], None) == code
    assert lib.inkling_dispatch_backward(d, *f[:6], None) == code
    assert lib.inkling_combine_forward(d, *f[:5], None) == code
    assert lib.inkling_combine_backward(d, *f[:6], None) == code


T, R, K, H = 100, 200, 2, 64
TOK, ROW, SLOT = T * H * 2, R * H * 4, T * K * 4
CALLS = {   # buffers in the order of the call, which of them are written, which may be NULL
    "inkling_dispatch_forward": (dict(x=TOK, positions=SLOT, weights=SLOT, rows=ROW), ("rows",), ("weights",)),
    "inkling_dispatch_backward": (dict(drows=ROW, positions=SLOT, weights=SLOT, x=TOK, dx=TOK, dweights=SLOT),
                                  ("dx", "dweights"), ("weights", "dweights")),
    "inkling_combine_forward": (dict(rows=ROW, positions=SLOT, weights=SLOT, addend=TOK, out=TOK), ("out",),
                                ("weights", "addend")),
    "inkling_combine_backward": (dict(dout=TOK, positions=SLOT, weights=SLOT, rows=ROW, drows=ROW, dweights=SLOT),
                                 ("drows", "dweights"), ("weights", "drows", "dweights")),
}


@pytest.mark.parametrize("name", CALLS)
def test_row_pointers(lib, name):
    sizes, written, optional = CALLS[name]
    d, at = ctypes.byref(_dispatch()), dict(zip(sizes, FAKE))
    call = lambda a, dd=d: getattr(lib, name)(dd, *a.values(), None)  # noqa: E731
    assert getattr(lib, name)(None, *at.values(), None) == BAD
    for n in sizes:
        if n not in optional:
            assert call(at | {n: None}) == BAD, n
        assert call(at | {n: at[n] + 2}) == BAD, n
        if n not in ("positions", "weights", "dweights"):
            assert call(at | {n: at[n] + 8}) == BAD, n
    for w, other in itertools.product(written, sizes):
        if w != other:
            for off in {0, 16, sizes[other] // 32 * 16, sizes[other] - 16}:
                assert call(at | {w: at[other] + off}) == BAD, (w, other, off)
            assert call(at | {other: at[w] + sizes[w] - 16}) == BAD, (w, other)
    assert call({n: None for n in sizes}, ctypes.byref(_dispatch(T=0))) == B.INKLING_OK
    if name == "inkling_combine_backward":
        assert call(at | {"drows": None, "dweights": None}) == BAD


def test_sizes_past_32_bits_are_value_errors():
    for make in (lambda v: B.make_order_dims(1, v, 2), lambda v: B.make_order_dims(1, 2, v),
                 lambda v: B.make_dispatch_dims(1, 1, v, 64, torch.float32, torch.float32),
                 lambda v: B._dispatch_plan(1, 1, 1, v, torch.float32, torch.float32)):
        for v in (2 ** 31, 2 ** 32 + 64, -2 ** 32 + 64):
            with pytest.raises(ValueError):
                make(v)


def test_binding_refuses_host_tensors_and_shapes():
    """Shapes are compared before a device is asked for."""
    x, pos = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        B.expert_order(torch.zeros((4,), dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        B.expert_order(pos.to(torch.int64), 4)
    with pytest.raises(ValueError):
        B.dispatch_forward(x, torch.zeros((5, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        B.dispatch_forward(x, pos, weights=torch.zeros((4, 3)))
    with pytest.raises(ValueError):
        B.dispatch_forward(x, pos.to(torch.int64))
    with pytest.raises(ValueError):
        B.dispatch_backward(x, pos, dweights=torch.zeros((4, 2)))
    with pytest.raises(ValueError):
        B.combine_backward(x, pos, dweights=torch.zeros((4, 2)))
    with pytest.raises(ValueError):
        B.combine_forward(x, pos, addend=torch.zeros((4, 9)))
    with pytest.raises(ValueError):
        B.combine_forward(torch.zeros((2, 4, 8)), pos)


def test_a_number_of_experts_changed_in_place_is_read_anew(monkeypatch):
    """A tensor as n_routed is its value at the call: sizes kept by the object would write past the results."""
    seen = []
    monkeypatch.setattr(B, "_operand", lambda *a: None)
    monkeypatch.setattr(B, "_call", lambda dev, name, dims, *a: seen.append(dims._obj.n_routed))
    topk, n = torch.zeros((4, 2), dtype=torch.int32), torch.tensor(200)
    for value in (200, 7, 300):
        n.fill_(value)
        o = B.expert_order(topk, n)
        assert seen[-1] == value and o["expert_counts"].shape == (value,) and o["expert_offsets"].shape == (value + 1,)
    for same in (8, 8.0, torch.tensor(8)):
        o = B.expert_order(topk, same)
        assert seen[-1] == 8 and o["expert_counts"].shape == (8,)
    with pytest.raises(TypeError):
        B.expert_order(topk, None)
