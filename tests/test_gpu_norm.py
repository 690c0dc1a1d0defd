"""Layer norm and RMS norm, forward and backward, against the formulas in 64 bits.

fp32 arithmetic: a thread adds at most 32 values one after another and the
workgroup's tree adds at most 22 more levels, so a sum of terms is off by at
most 64 2^-24 of the sum of their magnitudes.  With M = 64 2^-24 mean|x| for
the mean (its effect on the variance about it is of second order), the variance
and rstd are off by less than 2^-18 of themselves, and
  |dy| <= |w| rstd (M + 2^-17 |x - m|) + 2^-22 (|y| + |b|),
  |d dx| <= rstd 2^-17 (|c| + mean|c| + |xh| mean|c xh|),
  |d dw| <= (rows + 16) 2^-24 sum|dy xh|, and db likewise.
A bf16 result adds half a step, 2^-8 of the value.
"""
import sys

import numpy as np
import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(msg, file=sys.stderr, flush=True)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _make(R, H, dtype, seed=1, mean=0.3, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn((R, H), generator=g) * scale + mean).to(dtype).to(DEV),
            (1 + 0.3 * torch.randn((H,), generator=g)).to(DEV), (0.2 * torch.randn((H,), generator=g)).to(DEV),
            torch.randn((R, H), generator=g).to(dtype).to(DEV))


def _check(name, got, want, bound, dtype):
    got = _f64(got)
    bound = bound + (2.0 ** -8 * np.abs(want) if dtype == BF16 else 0.0) + 1e-30
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} off, worst {np.nanmax(np.abs(got - want) / bound):.2f} bounds, "
                           f"first at {np.argwhere(bad)[:3].tolist()}")


def _forward(x, w, b, eps, kind):
    m = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((x.shape[0], 1))
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps)
    y = (x - m) * r * w + b
    M = 64 * 2.0 ** -24 * np.abs(x).mean(1, keepdims=True) if kind == "layer" else 0.0
    tol = np.abs(w) * r * (M + 2.0 ** -17 * np.abs(x - m)) + 2.0 ** -22 * (np.abs(y) + np.abs(b))
    return m, r, y, M, tol


def _check_case(R, H, dtype, kind, mean=0.3, scale=2.0, eps=1e-6, seed=1):
    x, w, b, dy = _make(R, H, dtype, seed, mean, scale)
    layer = kind == "layer"
    out, stats = B.norm_forward(x, w, b if layer else None, eps=eps, kind=kind)
    r = B.norm_backward(dy, x, w, stats, kind=kind, bias=layer)
    torch.cuda.synchronize()
    x64, w64, d64 = _f64(x), _f64(w), _f64(dy)
    m, rs, y, M, tol = _forward(x64, w64, _f64(b) if layer else np.zeros(H), eps, kind)
    _check("out", out, y, tol, dtype)
    st = _f64(stats)
    assert (np.abs(st[:, :1] - m) <= M + 1e-30).all()
    assert (np.abs(st[:, 1:] - rs) <= 2.0 ** -18 * rs + rs ** 3 * (M ** 2)).all()
    # the backward takes the stats it is given
    m, rs = st[:, :1], st[:, 1:]
    xh = (x64 - m) * rs
    c = d64 * w64
    mc, mcx = c.mean(1, keepdims=True), (c * xh).mean(1, keepdims=True)
    dx = rs * (c - xh * mcx - (mc if layer else 0.0))
    _check("dx", r["dx"], dx, rs * 2.0 ** -17 * (np.abs(c) + np.abs(c).mean(1, keepdims=True) +
                                                np.abs(xh) * np.abs(c * xh).mean(1, keepdims=True)), dtype)
    n = (R + 16) * 2.0 ** -24
    _check("dweight", r["dweight"], (d64 * xh).sum(0), n * np.abs(d64 * xh).sum(0), F32)
    if layer:
        _check("dbias", r["dbias"], d64.sum(0), n * np.abs(d64).sum(0), F32)
    else:
        assert r["dbias"] is None


WIDTHS = [1, 3, 4, 8, 20, 100, 128, 512, 1000, 1024, 1028, 1237, 2048, 2056, 4096, 4098, 5000, 6144, 8192, 12288,
          16383, 16384]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, kind, dtype):
    _say(f"[norm] {H} {kind} {dtype}")
    _check_case(5, H, dtype, kind, seed=H)


@pytest.mark.parametrize("R,H", [(1, 6144), (2, 768), (17, 2048), (1000, 64), (9000, 40), (700, 1237)])
def test_row_counts(R, H):
    _check_case(R, H, BF16, "layer", seed=R)
    _check_case(R, H, F32, "rms", seed=R)


def test_large_mean_keeps_its_digits():
    """mean 1000 against a spread of 1: the variance is about the mean."""
    _check_case(6, 3000, F32, "layer", mean=1000.0, scale=1.0)


def test_wide_range():
    _check_case(6, 2048, F32, "layer", mean=0.0, scale=1e12)
    _check_case(6, 2048, F32, "rms", mean=0.0, scale=1e-12, eps=0.0)
    _check_case(6, 2048, BF16, "layer", mean=0.0, scale=1e-3, eps=1.0)


def test_constant_rows_and_non_finite_values():
    x, w, b, dy = _make(6, 520, F32, 3)
    x[1] = 7.5                                   # variance 0
    x[2, 5] = float("nan")
    x[3, 519] = float("inf")
    out, stats = B.norm_forward(x, w, b, eps=1e-6)
    r = B.norm_backward(dy, x, w, stats, bias=True)
    torch.cuda.synchronize()
    assert torch.equal(out[1], b)                # (x - mean) is exactly 0
    assert abs(float(stats[1, 1]) - 1e3) <= 1e-3
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    assert torch.isfinite(out[[0, 1, 4, 5]]).all() and torch.isfinite(r["dx"][[0, 1, 4, 5]]).all()
    assert torch.isnan(r["dx"][[2, 3]]).all() and torch.isnan(r["dweight"]).all()
    assert torch.isfinite(r["dbias"]).all()      # dout alone


def test_optional_parts():
    x, w, b, dy = _make(9, 1000, BF16, 4)
    out, stats = B.norm_forward(x, w, b)
    alone, none = B.norm_forward(x, w, b, save=False)
    assert none is None and torch.equal(alone, out)
    nob, _ = B.norm_forward(x, w)
    zero, _ = B.norm_forward(x, w, torch.zeros_like(b))
    assert torch.equal(nob, zero)
    full, part = B.norm_backward(dy, x, w, stats, bias=True), B.norm_backward(dy, x, w, stats)
    assert part["dbias"] is None and torch.equal(full["dx"], part["dx"])
    assert torch.equal(full["dweight"], part["dweight"])


def test_no_rows():
    x, w, b, dy = _make(4, 200, BF16, 5)
    out, stats = B.norm_forward(x[:0], w, b)
    assert out.shape == (0, 200) and stats.shape == (0, 2)
    mark = dict(dweight=torch.full((200,), 9.0, device=DEV), dbias=torch.full((200,), 9.0, device=DEV))
    r = B.norm_backward(dy[:0], x[:0], w, stats, **mark)
    torch.cuda.synchronize()
    assert int(r["dweight"].count_nonzero()) == 0 and int(r["dbias"].count_nonzero()) == 0


def test_gradients_against_differences():
    """Central differences in 64 bits of <dout, y(x, w, b)>."""
    R, H, eps = 3, 24, 1e-3
    for kind in ("layer", "rms"):
        x, w, b, dy = _make(R, H, F32, 6)
        b0 = _f64(b) if kind == "layer" else np.zeros(H)
        _, stats = B.norm_forward(x, w, b if kind == "layer" else None, eps=eps, kind=kind)
        r = B.norm_backward(dy, x, w, stats, kind=kind, bias=kind == "layer")
        torch.cuda.synchronize()
        x0, w0, d = _f64(x), _f64(w), _f64(dy)
        f = lambda xx, ww, bb: float((d * _forward(xx, ww, bb, eps, kind)[2]).sum())  # noqa: E731
        step, g = 1e-5, np.random.default_rng(2)
        for _ in range(8):
            v = g.standard_normal((R, H))
            num = (f(x0 + step * v, w0, b0) - f(x0 - step * v, w0, b0)) / (2 * step)
            assert abs(num - (_f64(r["dx"]) * v).sum()) <= 1e-4
            v = g.standard_normal(H)
            num = (f(x0, w0 + step * v, b0) - f(x0, w0 - step * v, b0)) / (2 * step)
            assert abs(num - (_f64(r["dweight"]) * v).sum()) <= 1e-4
            if kind == "layer":
                num = (f(x0, w0, b0 + step * v) - f(x0, w0, b0 - step * v)) / (2 * step)
                assert abs(num - (_f64(r["dbias"]) * v).sum()) <= 1e-4


def test_two_graphs_that_share_a_workspace_and_a_side_stream():
    cases = [_make(70, 1000, BF16, 7), _make(33, 2056, BF16, 8)]
    ws = torch.empty(max(B.norm_backward_workspace_size(B.make_norm_dims(70, 1000, "layer", BF16, 0.0)),
                         B.norm_backward_workspace_size(B.make_norm_dims(33, 2056, "layer", BF16, 0.0))),
                     dtype=torch.uint8, device=DEV)
    graphs = []
    for x, w, b, dy in cases:
        bufs = dict(dx=torch.zeros_like(x), dweight=torch.zeros_like(w), dbias=torch.zeros_like(w))
        out, stats = torch.zeros_like(x), torch.zeros((x.shape[0], 2), device=DEV)

        def step(x=x, w=w, b=b, dy=dy, bufs=bufs, out=out, stats=stats):
            B.norm_forward(x, w, b, out=out, stats=stats)
            B.norm_backward(dy, x, w, stats, workspace=ws, **bufs)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, bufs, out, stats))
    for turn in range(3):
        for (x, w, b, dy), (g, bufs, out, stats) in zip(cases, graphs):
            for t in (out, stats, *bufs.values()):
                t.fill_(-3.0)
            g.replay()
            torch.cuda.synchronize()
            o, s = B.norm_forward(x, w, b)
            r = B.norm_backward(dy, x, w, s, bias=True)
            torch.cuda.synchronize()
            assert torch.equal(out, o) and torch.equal(stats, s), f"turn {turn}"
            for k in bufs:
                assert torch.equal(bufs[k], r[k]), f"turn {turn}: {k}"


def test_element_offsets_past_32_bits():
    H = 4100                                          # rows of single bf16 values: not whole vectors of 8
    R = (1 << 32) // H // 2 + 50                      # byte offsets past 2^32, elements past 2^31
    x = torch.ones((R, H), dtype=BF16, device=DEV)
    x[:, ::2] = -1.0
    tail, w, b, dy = _make(8, H, BF16, 9)
    x[-8:] = tail
    out, stats = B.norm_forward(x, w, b)
    want, st = B.norm_forward(tail, w, b)
    assert torch.equal(out[-8:], want) and torch.equal(stats[-8:], st)
    d = torch.zeros((R, H), dtype=BF16, device=DEV)
    d[-8:] = dy
    del out
    r, r2 = B.norm_backward(d, x, w, stats, bias=True), B.norm_backward(dy, tail, w, st, bias=True)
    torch.cuda.synchronize()
    assert torch.equal(r["dx"][-8:], r2["dx"]) and int(r["dx"][:-8].count_nonzero()) == 0
    # the same 8 terms, in another order with zeros between
    assert bool(((r["dweight"] - r2["dweight"]).abs() <= 16 * 2.0 ** -24 * 8 * 60).all())


def test_refusals():
    x, w, b, dy = _make(10, 64, BF16, 10)
    _, stats = B.norm_forward(x, w, b)
    for bad in (dict(x=x.half()), dict(x=x.cpu()), dict(x=x[:, :32]), dict(weight=w.to(BF16)), dict(bias=b[:5]),
                dict(kind="batch"), dict(out=x.float()), dict(stats=stats[:5]), dict(save=False, stats=stats)):
        with pytest.raises(ValueError):
            B.norm_forward(**(dict(x=x, weight=w, bias=b) | bad))
    for bad in (dict(kind="rms"), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(out=x)):
        with pytest.raises(B.InklingError) as e:
            B.norm_forward(**(dict(x=x, weight=w, bias=b) | bad))
        assert e.value.code == B.INKLING_ERR_INVALID_ARGUMENT
    wide = torch.zeros((1, 16385), dtype=BF16, device=DEV)
    with pytest.raises(B.InklingError) as e:
        B.norm_forward(wide, torch.ones(16385, device=DEV))
    assert e.value.code == B.INKLING_ERR_UNSUPPORTED
    for bad in (dict(dout=dy.float()), dict(dout=dy[:5]), dict(stats=stats[:5]), dict(dweight=w[:5])):
        with pytest.raises(ValueError):
            B.norm_backward(**(dict(dout=dy, x=x, weight=w, stats=stats) | bad))
    with pytest.raises(B.InklingError) as e:
        B.norm_backward(dy, x, w, stats, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == B.INKLING_ERR_WORKSPACE
    with pytest.raises(B.InklingError) as e:
        B.norm_backward(dy, x, w, stats, dx=x)
    assert e.value.code == B.INKLING_ERR_INVALID_ARGUMENT
