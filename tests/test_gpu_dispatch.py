"""Tokens sorted by expert and back against the definitions in 64 bits.

The order is compared number by number.  Copies (no weights, one type) have to be
equal.  Otherwise fp32 arithmetic of unit roundoff u = 2^-24: a product is off by u
of itself; a gather's sum of n terms in sequence by at most (n + 1) u of the sum of
their sizes; of a weights' gradient, every product passes its own rounding and at
most H / 256 + 32 sums (columns of a lane's vectors, its vectors, 64 lanes, 4
waves).  A bf16 result adds half a step, 2^-8 of the value.
"""
import sys

import numpy as np
import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
MARK = -777.0


def _say(msg):
    print(msg, file=sys.stderr, flush=True)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _half_step(dtype):
    return 2.0 ** -8 if dtype == BF16 else 0.0


# ---- the order -------------------------------------------------------------------------


def _ref_order(topk, E, mask=None):
    T, k = topk.shape
    key = np.where((topk >= 0) & (topk < E), topk, E)
    if mask is not None:
        key = np.where(mask[:, None] != 0, E, key)
    key = key.reshape(-1)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)[:E]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    used = offsets[-1]
    slots = np.full(T * k, -1)
    slots[:used] = order[:used]
    pos = np.full(T * k, -1)
    pos[order[:used]] = np.arange(used)
    return counts, offsets, slots, pos.reshape(T, k)


def _check_order(got, want):
    for name, w in zip(("expert_counts", "expert_offsets", "sorted_slots", "positions"), want):
        assert np.array_equal(got[name].cpu().numpy(), w), name


@pytest.mark.parametrize("T,E,k,kind", [
    (1, 1, 1, "any"), (1, 8, 2, "any"), (63, 5, 1, "any"), (64, 64, 3, "any"), (65, 65, 8, "any"),
    (32, 128, 8, "distinct"), (1024, 128, 8, "distinct"),      # the most that one workgroup takes
    (8193, 128, 1, "distinct"), (1025, 100, 8, "distinct"),    # the fewest that take two launches
    (8192, 128, 8, "distinct"), (5000, 512, 32, "any"), (40000, 512, 8, "any"), (33333, 511, 7, "any"),
    (3000, 256, 4, "one"), (700, 3, 2, "one"), (2500, 129, 6, "outside"), (300, 12, 5, "outside"),
    (70000, 2, 8, "any"),
])
@pytest.mark.parametrize("masked", [False, True])
def test_order(T, E, k, kind, masked):
    _say(f"order T={T} E={E} k={k} {kind} masked={masked}")
    rng = np.random.default_rng(T * 31 + E * 7 + k)
    if kind == "distinct":
        topk = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    elif kind == "one":          # every slot to one expert, the same one twice in a token
        topk = np.full((T, k), E - 1)
    elif kind == "outside":
        topk = rng.integers(-3, E + 3, (T, k))
        topk[rng.random((T, k)) < 0.05] = -2 ** 31
        topk[rng.random((T, k)) < 0.05] = 2 ** 31 - 1
    else:
        topk = rng.integers(0, E, (T, k))
    mask = (rng.random(T) < 0.3).astype(np.uint8) * rng.integers(1, 256, T).astype(np.uint8) if masked else None
    t = torch.from_numpy(topk.astype(np.int32)).to(DEV)
    m = None if mask is None else torch.from_numpy(mask).to(DEV)
    got = B.expert_order(t, E, padding_mask=m)
    _check_order(got, _ref_order(topk, E, mask))


def test_order_of_the_most_slots():
    """Nearly 2^31 slots: every slot in its row, rows by expert, then by slot."""
    T, E, k = 71582000, 5, 30
    n = T * k
    _say(f"order of {n} slots")
    topk = torch.randint(0, E + 1, (T, k), dtype=torch.int32, device=DEV)     # E: no row
    got = B.expert_order(topk, E)
    flat, pos, slots = topk.view(-1), got["positions"].view(-1), got["sorted_slots"]
    ends = got["expert_offsets"].tolist()
    assert ends[0] == 0 and np.diff(ends).tolist() == got["expert_counts"].tolist()
    used, step, rows = ends[-1], 1 << 26, 0
    for a in range(0, n, step):
        p, e = pos[a:a + step], flat[a:a + step]
        has = e < E
        assert torch.equal(p >= 0, has)
        at = has.nonzero().view(-1)
        rows += at.numel()
        assert torch.equal(slots[p[at].long()].long(), at + a)
    assert rows == used and bool((slots[used:used + (1 << 20)] == -1).all()) and int(slots[n - 1]) == -1
    for a in range(0, used - 1, step):
        c = slots[a:min(a + step + 1, used)].long()
        key = flat[c].long() * n + c
        assert bool((key[1:] > key[:-1]).all())
    for e in range(E):
        assert int(flat[slots[ends[e]].long()]) == e and int(flat[slots[ends[e + 1] - 1].long()]) == e


def test_order_of_nothing():
    got = B.expert_order(torch.empty((0, 4), dtype=torch.int32, device=DEV), 7)
    assert got["expert_offsets"].tolist() == [0] * 8 and got["expert_counts"].tolist() == [0] * 7
    t = torch.randint(0, 7, (50, 4), dtype=torch.int32, device=DEV)
    got = B.expert_order(t, 7, padding_mask=torch.ones(50, dtype=torch.uint8, device=DEV))
    assert got["expert_offsets"].tolist() == [0] * 8
    assert bool((got["sorted_slots"] == -1).all()) and bool((got["positions"] == -1).all())


def test_order_agrees_with_the_router():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((300, 64), generator=g).to(BF16).to(DEV)
    bank, bias = torch.randn((20, 64), generator=g).to(DEV), torch.zeros(16, device=DEV)
    mask = (torch.rand(300, generator=g) < 0.2).to(torch.uint8).to(DEV)
    r = B.route(x, bank, bias, 4, 1.0, 1.0, padding_mask=mask)
    o = B.expert_order(r["topk_indices"], 16, padding_mask=mask)
    used = int(o["expert_offsets"][-1])
    assert torch.equal(o["expert_offsets"], r["expert_offsets"])
    assert torch.equal(o["expert_counts"], r["expert_counts"])
    assert torch.equal(o["sorted_slots"][:used], r["sorted_slots"][:used])


# ---- rows and tokens ---------------------------------------------------------------------

SHAPES = [   # T, E, k, H
    (1, 4, 1, 1), (3, 4, 2, 3), (5, 4, 4, 7), (17, 8, 8, 8), (9, 8, 3, 9), (33, 8, 2, 64), (20, 16, 5, 65),
    (7, 16, 9, 127), (13, 16, 16, 128), (11, 40, 32, 129), (30, 12, 2, 512), (6, 12, 8, 513), (25, 12, 2, 1237),
    (4, 128, 8, 6144), (10, 64, 6, 2048), (2, 4, 3, 16391),
]
TYPES = [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)]


def _positions(T, E, k, seed, drop=0.1, pad=0.1):
    rng = np.random.default_rng(seed)
    topk = rng.integers(0, E, (T, k))
    topk[rng.random((T, k)) < drop] = -1
    mask = (rng.random(T) < pad).astype(np.uint8)
    _, offsets, _, pos = _ref_order(topk, E, mask)
    return pos, int(offsets[-1])


def _randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def _case(T, E, k, H, token, rows):
    pos, used = _positions(T, E, k, T * 13 + k)
    w = _randn((T, k), F32, 3)
    return (pos, used, torch.from_numpy(pos.astype(np.int32)).to(DEV), w, _randn((T, H), token, 1),
            _randn((T * k, H), rows, 2))


def _close(name, got, want, bound):
    bad = ~(np.abs(_f64(got) - want) <= bound)
    assert not bad.any(), f"{name}: {int(bad.sum())} off, first at {np.argwhere(bad)[:3].tolist()}"


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("token,rows", TYPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_forward(T, E, k, H, token, rows, weighted):
    _say(f"dispatch_forward {T} {E} {k} {H} {token} {rows} {weighted}")
    pos, used, p, w, x, _ = _case(T, E, k, H, token, rows)
    out = torch.full((T * k, H), MARK, dtype=rows, device=DEV)
    assert B.dispatch_forward(x, p, weights=w if weighted else None, rows=out) is out
    want = np.full((T * k, H), MARK)
    t, i = np.nonzero(pos >= 0)
    want[pos[t, i]] = _f64(x)[t] * (_f64(w)[t, i][:, None] if weighted else 1.0)
    _close("rows", out[:used], want[:used], np.abs(want[:used]) * ((U if weighted else 0.0) +
           (0.0 if not weighted and (rows == token or rows == F32) else _half_step(rows) * (1.0 + U))))
    assert bool((out[used:] == torch.tensor(MARK, dtype=rows)).all()), "a row that no position names"


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("token,rows", TYPES)
@pytest.mark.parametrize("weighted,added", [(False, False), (True, True), (True, False)])
def test_combine_forward(T, E, k, H, token, rows, weighted, added):
    _say(f"combine_forward {T} {E} {k} {H} {token} {rows} {weighted} {added}")
    pos, used, p, w, x, y = _case(T, E, k, H, token, rows)
    y[used:] = float("nan")      # rows that no position names
    out = B.combine_forward(y, p, weights=w if weighted else None, addend=x if added else None, out_dtype=token)
    assert out.dtype == token
    terms = np.zeros((T, k + 1, H))
    if added:
        terms[:, 0] = _f64(x)
    t, i = np.nonzero(pos >= 0)
    terms[t, 1 + i] = _f64(y)[pos[t, i]] * (_f64(w)[t, i][:, None] if weighted else 1.0)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    err = (k + 2) * U * size
    _close("out", out, want, err + _half_step(token) * (np.abs(want) + err))


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("token,rows", TYPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_gradients(T, E, k, H, token, rows, weighted):
    """Both operators' gradients against the formulas."""
    _say(f"gradients {T} {E} {k} {H} {token} {rows} {weighted}")
    pos, used, p, w, x, y = _case(T, E, k, H, token, rows)
    ww = w if weighted else None
    t, i = np.nonzero(pos >= 0)
    wn = _f64(w) if weighted else np.ones((T, k))
    xn, yn = _f64(x), _f64(y)
    dots, sizes = np.zeros((T, k)), np.zeros((T, k))
    prod = xn[t] * yn[pos[t, i]]
    dots[t, i], sizes[t, i] = prod.sum(1), np.abs(prod).sum(1)
    dw_bound = (H / 256 + 33) * U * sizes
    y[used:] = float("inf")
    # combine: dout = x, rows = y
    drows = torch.full((T * k, H), MARK, dtype=rows, device=DEV)
    g = B.combine_backward(x, p, rows=y, weights=ww, drows=drows)
    want = xn[t] * wn[t, i][:, None]
    at = pos[t, i]
    _close("drows", g["drows"][torch.from_numpy(at).to(DEV)], want, np.abs(want) * (U + _half_step(rows) * (1 + U)))
    assert bool((drows[used:] == torch.tensor(MARK, dtype=rows)).all())
    _close("dweights of the combine", g["dweights"], dots, dw_bound)
    g0 = B.combine_backward(x, p, weights=ww, drows=torch.full_like(drows, MARK))
    assert g0["dweights"] is None and torch.equal(g0["drows"], drows)
    # dispatch: x = x, drows = y
    terms = np.zeros((T, k, H))
    terms[t, i] = yn[at] * wn[t, i][:, None]
    want, size = terms.sum(1), np.abs(terms).sum(1)
    err = (k + 2) * U * size
    g = B.dispatch_backward(y, p, weights=ww, x=x)
    _close("dx", g["dx"], want, err + _half_step(token) * (np.abs(want) + err))
    _close("dweights of the dispatch", g["dweights"], dots, dw_bound)
    g0 = B.dispatch_backward(y, p, weights=ww, dx_dtype=token)
    assert g0["dweights"] is None and torch.equal(g0["dx"], g["dx"])


def test_gradients_are_the_differences():
    """<v, combine> and <v, dispatch> moved along a direction, in fp32: both are linear in rows, in x and in the
    weights, so central differences are exact but for rounding: n = 40 results of at most 4 terms, each product of
    magnitude below 40, differences over a step of 1: below 40 * 300 * 2^-24 * 40 = 0.03."""
    T, E, k, H = 6, 4, 3, 20
    pos, used, p, w, x, y = _case(T, E, k, H, F32, F32)
    v, vr = _randn((T, H), F32, 8), _randn((T * k, H), F32, 9)
    vr[used:] = 0.0
    y[used:] = 0.0
    gc, gd = B.combine_backward(v, p, rows=y, weights=w, drows=torch.zeros_like(y)), B.dispatch_backward(
        vr, p, weights=w, x=x)
    dy, dw, dx = _randn(y.shape, F32, 10), _randn(w.shape, F32, 11), _randn(x.shape, F32, 12)
    combine = lambda yy, ww: float((B.combine_forward(yy, p, weights=ww).double() * v.double()).sum())  # noqa: E731
    dispatch = lambda xx, ww: float((B.dispatch_forward(xx, p, weights=ww, rows=torch.zeros_like(y)).double() *  # noqa: E731
                                     vr.double()).sum())
    for fd, grad, step in ((combine(y + dy, w) - combine(y - dy, w), gc["drows"], dy),
                           (combine(y, w + dw) - combine(y, w - dw), gc["dweights"], dw),
                           (dispatch(x + dx, w) - dispatch(x - dx, w), gd["dx"], dx),
                           (dispatch(x, w + dw) - dispatch(x, w - dw), gd["dweights"], dw)):
        assert abs(fd / 2 - float((grad.double() * step.double()).sum())) < 0.03


def test_fewer_rows_than_slots():
    """Positions past the buffer are dropped: not written, not read, no gradient."""
    T, E, k, H = 40, 4, 2, 96
    pos, used, p, w, x, y = _case(T, E, k, H, BF16, BF16)
    n = used // 2
    guard = torch.full((T * k, H), MARK, dtype=BF16, device=DEV)
    B.dispatch_forward(x, p, rows=guard[:n])
    assert bool((guard[n:] == MARK).all())
    cut = torch.where(p < n, p, -1)
    full = B.dispatch_forward(x, cut, rows=torch.full_like(guard, MARK))
    assert torch.equal(full[:n], guard[:n])
    assert torch.equal(B.combine_forward(y[:n], p, weights=w), B.combine_forward(y, cut, weights=w))
    a, b = B.combine_backward(x, p, rows=y[:n].contiguous(), weights=w), B.combine_backward(x, cut, rows=y, weights=w)
    assert torch.equal(a["dweights"], b["dweights"]) and torch.equal(a["drows"], b["drows"][:n])
    bad = p.clone()
    bad[0, 0], bad[1, 0], bad[2, 0] = -5, 2 ** 31 - 1, T * k
    ok = p.clone()
    ok[0, 0] = ok[1, 0] = ok[2, 0] = -1
    assert torch.equal(B.combine_forward(y, bad), B.combine_forward(y, ok))


def test_no_rows_and_no_tokens():
    x, p = _randn((5, 40), F32, 1), torch.zeros((5, 2), dtype=torch.int32, device=DEV)
    none = torch.empty((0, 40), device=DEV)
    assert torch.equal(B.combine_forward(none, p, addend=x), x)
    assert bool((B.combine_forward(none, p) == 0).all())
    g = B.dispatch_backward(none, p, x=x)
    assert bool((g["dx"] == 0).all()) and bool((g["dweights"] == 0).all())
    g = B.combine_backward(x, p, rows=none)
    assert g["drows"].shape == (0, 40) and bool((g["dweights"] == 0).all())
    assert B.dispatch_forward(x, p, rows=none) is none
    assert B.combine_backward(x, p, drows=none)["drows"] is none
    e = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    assert B.combine_forward(_randn((3, 40), F32, 1), e).shape == (0, 40)
    assert B.dispatch_forward(none, e).shape == (0, 40)


def test_infinities_and_nan():
    x = torch.ones((4, 24), device=DEV)
    x[0, 3], x[1, 5], x[2, 23] = float("inf"), float("nan"), float("-inf")
    p = torch.tensor([[0, 1], [2, -1], [3, 4], [-1, -1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.0, 2.0], [1.0, float("nan")], [-1.0, 1.0], [float("inf"), 1.0]], device=DEV)
    for dt in (F32, BF16):
        r = B.dispatch_forward(x, p, weights=w, rows=torch.zeros((8, 24), dtype=dt, device=DEV))
        assert bool(r[0, 3].isnan()) and float(r[1, 3]) == float("inf") and bool(r[2, 5].isnan())
        assert float(r[3, 23]) == float("inf") and float(r[4, 23]) == float("-inf")
        out = B.combine_forward(r, p, weights=w.nan_to_num(1.0, 1.0, 1.0))
        assert bool(out[0, 3].isnan()) and bool(out[1, 5].isnan()) and float(out[2, 23]) == float("-inf")
        assert bool((out[3] == 0).all()), "a dropped slot's weight has no part"
        assert int(out.isfinite().sum()) == 4 * 24 - 3
    g = B.combine_backward(x, p, rows=torch.ones((8, 24), device=DEV), weights=w,
                           drows=torch.zeros((8, 24), device=DEV))
    assert g["dweights"][0].tolist() == [float("inf")] * 2 and bool(g["dweights"][1, 0].isnan())
    assert float(g["dweights"][1, 1]) == 0.0 and g["dweights"][3].tolist() == [0.0, 0.0]


def test_past_32_bits():
    """Rows that begin past 2^32 bytes and past 2^31 values."""
    T, k, H = 51200, 8, 6144
    rows = torch.empty((T * k, H), dtype=BF16, device=DEV)
    x = _randn((64, H), BF16, 4).repeat(T // 64, 1)
    pos = (torch.arange(T * k, device=DEV, dtype=torch.int32).reshape(k, T).t()).contiguous()   # row i T + t
    B.dispatch_forward(x, pos, rows=rows)
    for i in range(k):
        assert torch.equal(rows[i * T:(i + 1) * T], x), i
    out = B.combine_forward(rows, pos, weights=torch.full((T, k), 0.125, device=DEV))
    assert torch.equal(out, x)
    rows.zero_()
    g = B.combine_backward(x, pos, weights=torch.full((T, k), 2.0, device=DEV), drows=rows)
    for i in range(k):
        assert torch.equal(rows[i * T:(i + 1) * T], 2 * x), i
    g = B.dispatch_backward(rows, pos, x=x)
    assert torch.equal(g["dx"], 16 * x)


def test_the_run_of_an_expert_block():
    """Order, dispatch, products, activation, combine and all of it back, against the layer in 64 bits."""
    T, E, k, H, I = 70, 8, 2, 64, 32
    rng = np.random.default_rng(2)
    topk = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    x, wu, wd = _randn((T, H), F32, 1), _randn((E, 2 * I, H), F32, 2, 0.2), _randn((E, H, I), F32, 3, 0.2)
    w, dout = _randn((T, k), F32, 4).abs(), _randn((T, H), F32, 5)
    o = B.expert_order(torch.from_numpy(topk).to(DEV), E)
    off, pos = o["expert_offsets"], o["positions"]
    rows = B.dispatch_forward(x, pos)
    act, _ = B.swiglu_forward(B.grouped_linear(rows, wu, off), save=False)
    y = B.grouped_linear(act, wd, off)
    out = B.combine_forward(y, pos, weights=w, addend=x)
    g = B.combine_backward(dout, pos, rows=y, weights=w)
    dwd = B.grouped_weight_grad(g["drows"], act, off)
    # 64 bits, token by token
    X, U_, D, W, DO = (t.double().cpu() for t in (x, wu, wd, w, dout))
    want, dww, dD = X.clone(), torch.zeros((T, k), dtype=torch.float64), torch.zeros_like(D)
    for t in range(T):
        for i in range(k):
            e = int(topk[t, i])
            h = U_[e] @ X[t]
            a = torch.nn.functional.silu(h[0::2]) * h[1::2]
            z = D[e] @ a
            want[t] += W[t, i] * z
            dww[t, i] = DO[t] @ z
            dD[e] += W[t, i] * torch.outer(DO[t], a)
    for name, got, ref in (("out", out, want), ("dweights", g["dweights"], dww), ("dW", dwd, dD)):
        err = float((got.cpu().double() - ref).abs().max())
        # sums of at most 64 products through two projections, fp32: 200 roundings of the largest value
        assert err <= 400 * U * float(ref.abs().max()), (name, err)


# ---- streams, graphs, repeats ----------------------------------------------------------------


def test_repeats_bit_for_bit_and_on_another_stream():
    T, E, k, H = 3000, 100, 8, 1237
    pos, used, p, w, x, y = _case(T, E, k, H, BF16, BF16)
    topk = torch.randint(0, E, (T, k), dtype=torch.int32, device=DEV)
    a = [B.combine_forward(y, p, weights=w), B.combine_backward(x, p, rows=y, weights=w)["dweights"],
         B.dispatch_backward(y, p, weights=w, x=x)["dx"], *B.expert_order(topk, E).values()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = [B.combine_forward(y, p, weights=w), B.combine_backward(x, p, rows=y, weights=w)["dweights"],
             B.dispatch_backward(y, p, weights=w, x=x)["dx"], *B.expert_order(topk, E).values()]
    s.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T", [48, 2000])
def test_captured(T):
    """A step in a graph, replayed with new inputs in the same buffers, eager work between the replays."""
    E, k, H = 16, 6, 520
    topk = torch.randint(0, E, (T, k), dtype=torch.int32, device=DEV)
    x, w = _randn((T, H), BF16, 1), _randn((T, k), F32, 2)
    n = B.expert_order_workspace_size(B.make_order_dims(T, E, k))
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)

    def step(ws, bufs):
        o = B.expert_order(topk, E, workspace=ws, **bufs["order"])
        rows = B.dispatch_forward(x, o["positions"], rows=bufs["rows"])
        out = B.combine_forward(rows, o["positions"], weights=w, addend=x, out=bufs["out"])
        g = B.combine_backward(out, o["positions"], rows=rows, weights=w, drows=bufs["drows"], dweights=bufs["dw"])
        B.dispatch_backward(g["drows"], o["positions"], dx=bufs["dx"])

    def buffers():
        i32 = dict(dtype=torch.int32, device=DEV)
        return {"order": {"expert_counts": torch.empty(E, **i32), "expert_offsets": torch.empty(E + 1, **i32),
                          "sorted_slots": torch.empty(T * k, **i32), "positions": torch.empty((T, k), **i32)},
                "rows": torch.zeros((T * k, H), dtype=BF16, device=DEV), "out": torch.empty_like(x),
                "drows": torch.zeros((T * k, H), dtype=BF16, device=DEV), "dw": torch.empty_like(w),
                "dx": torch.empty_like(x)}

    held, eager = buffers(), buffers()
    step(ws, held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ws, held)
    for turn in range(4):
        topk.copy_(torch.randint(-1, E, (T, k), dtype=torch.int32, device=DEV))
        x.copy_(_randn((T, H), BF16, 20 + turn))
        for b in (held, eager):
            b["rows"].zero_()
            b["drows"].zero_()
        graph.replay()
        step(None, eager)
        torch.cuda.synchronize()
        for n in ("rows", "out", "drows", "dw", "dx"):
            assert torch.equal(held[n], eager[n]), (turn, n)
        for n in held["order"]:
            assert torch.equal(held["order"][n], eager["order"][n]), (turn, n)


def test_binding_refusals():
    x, p = _randn((4, 16), F32, 1), torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    r = _randn((8, 16), F32, 2)
    with pytest.raises(ValueError):
        B.dispatch_forward(x, p.cpu())
    with pytest.raises(ValueError):
        B.dispatch_forward(x.t(), p)
    with pytest.raises(ValueError):
        B.dispatch_forward(x, p, rows=r[:, :8])
    with pytest.raises(ValueError):
        B.dispatch_forward(x, p, rows=r, rows_dtype=BF16)
    with pytest.raises(ValueError):
        B.combine_forward(r, p, addend=x.to(BF16), out_dtype=F32)
    with pytest.raises(ValueError):
        B.combine_forward(r, p, out=torch.empty((5, 16), device=DEV))
    with pytest.raises(ValueError):
        B.dispatch_backward(r, p, x=x, dx_dtype=BF16)
    with pytest.raises(ValueError):
        B.combine_backward(x, p, rows=r, drows=torch.empty((7, 16), device=DEV))
    with pytest.raises(ValueError):
        B.expert_order(p, 4, padding_mask=torch.zeros(3, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        B.expert_order(p, 4, positions=torch.empty((4, 3), dtype=torch.int32, device=DEV))
    with pytest.raises(B.InklingError):
        B.expert_order(p, 513)
    with pytest.raises(B.InklingError) as e:
        B.combine_forward(r, p, addend=x, out=x)
    assert e.value.code == B.INKLING_ERR_INVALID_ARGUMENT


# ---- results that a C caller does not want -------------------------------------------------


@pytest.mark.parametrize("T,E,k", [(50, 7, 3), (1024, 128, 8), (9000, 128, 8), (3000, 512, 32), (0, 5, 2)])
@pytest.mark.parametrize("without", [("expert_counts",), ("sorted_slots",), ("expert_counts", "sorted_slots")])
def test_order_without_some_results(T, E, k, without):
    """expert_counts and sorted_slots may be NULL, in one launch and in two: the others are the same."""
    _say(f"order T={T} E={E} k={k} without {without}")
    rng = np.random.default_rng(T + k)
    topk = torch.from_numpy(rng.integers(-1, E + 1, (T, k)).astype(np.int32)).to(DEV)
    mask = torch.from_numpy((rng.random(T) < 0.2).astype(np.uint8)).to(DEV)
    want = B.expert_order(topk, E, padding_mask=mask)
    got = {n: torch.full_like(t, -9) for n, t in want.items()}
    dims, need = B._order_plan(T, E, k)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    at = [None if n in without else got[n].data_ptr() for n in ("expert_counts", "expert_offsets", "sorted_slots",
                                                                "positions")]
    B._call(torch.device(DEV), "inkling_expert_order", dims, topk.data_ptr(), mask.data_ptr(), *at, ws.data_ptr(), need)
    for n in want:
        assert bool((got[n] == -9).all()) if n in without else torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("k", [1, 3, 8, 9, 17])
@pytest.mark.parametrize("H", [5, 64, 500, 1237, 2056])      # 16 lanes, a wave and a workgroup a token
@pytest.mark.parametrize("token_dtype,rows_dtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_combine_backward_of_the_weights_alone(k, H, token_dtype, rows_dtype):
    """drows may be NULL: dweights are the same, bit by bit."""
    _say(f"combine_backward without drows k={k} H={H} {token_dtype} {rows_dtype}")
    T, E = 37, 20
    g = torch.Generator().manual_seed(k * H)
    topk = torch.randint(-1, E, (T, k), generator=g).to(torch.int32).to(DEV)
    pos = B.expert_order(topk, E)["positions"]
    dout = torch.randn((T, H), generator=g).to(token_dtype).to(DEV)
    rows = torch.randn((T * k, H), generator=g).to(rows_dtype).to(DEV)
    w = torch.rand((T, k), generator=g).to(DEV)
    want = B.combine_backward(dout, pos, rows=rows, weights=w)["dweights"]
    got = torch.full((T, k), MARK, device=DEV)
    B._call(torch.device(DEV), "inkling_combine_backward", B._dispatch_plan(T, T * k, k, H, token_dtype, rows_dtype),
            dout.data_ptr(), pos.data_ptr(), w.data_ptr(), rows.data_ptr(), None, got.data_ptr())
    assert torch.equal(got, want) and bool((want != 0).any())
