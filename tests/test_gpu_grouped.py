"""Products grouped by expert (inkling_grouped_linear, _input_grad, _weight_grad)
against sums in 64 bits.

Tolerance of a value v = sum of n products: the products of two bf16 are exact
in fp32 and those of two fp32 are rounded once (2^-24 of the product); adding n
terms in fp32 in any order moves the sum by at most n 2^-24 sum|products| to
first order.  Twice that covers the second order (n 2^-24 < 2^-9 here) and
matrix instructions that round their inner sums toward zero (one step, 2^-23,
an addition).  A bf16 result adds half a step, 2^-8 |v|.
"""
import sys

import numpy as np
import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
MARK = -777.0   # what result buffers hold before a call (exact in bf16)


def _say(msg):
    print(msg, file=sys.stderr, flush=True)


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _close(name, got, want, absum, n, dtype):
    got = _f64(got)
    bound = (2 * n * 2.0 ** -24) * absum + (2.0 ** -8 * np.abs(want) if dtype == BF16 else 0.0) + 1e-30
    bad = np.abs(got - want) > bound
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} values off, worst "
                           f"{float(np.max(np.abs(got - want) / bound)):.2f} bounds at {np.argwhere(bad)[:3].tolist()}")


class Case:
    def __init__(self, counts, K, N, dtype, first=0, room=0, tokens=None, seed=1):
        self.counts, self.K, self.N, self.dtype = counts, K, N, dtype
        ends = np.cumsum([first] + list(counts))
        self.ends = ends
        self.R = int(ends[-1]) + room
        self.offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
        g = np.random.default_rng(seed)
        self.index = None if tokens is None else torch.tensor(g.integers(0, tokens, self.R), dtype=torch.int32,
                                                              device=DEV)
        self.x = _rand((self.R if tokens is None else tokens, K), dtype, seed + 1)
        self.w = _rand((len(counts), N, K), dtype, seed + 2, 0.1)
        self.dout = _rand((self.R, N), dtype, seed + 3)

    def rows(self, e):
        return slice(int(self.ends[e]), int(self.ends[e + 1]))

    def x_rows(self):
        x = _f64(self.x)
        return x if self.index is None else x[self.index.cpu().numpy()]

    def live(self):
        m = np.zeros(self.R, bool)
        m[int(self.ends[0]):int(self.ends[-1])] = True
        return m

    def forward(self):
        x, w = self.x_rows(), _f64(self.w)
        out, ab = np.full((self.R, self.N), MARK), np.zeros((self.R, self.N))
        for e in range(len(self.counts)):
            out[self.rows(e)] = x[self.rows(e)] @ w[e].T
            ab[self.rows(e)] = np.abs(x[self.rows(e)]) @ np.abs(w[e]).T
        return out, ab

    def input_grad(self):
        d, w = _f64(self.dout), _f64(self.w)
        out, ab = np.full((self.R, self.K), MARK), np.zeros((self.R, self.K))
        for e in range(len(self.counts)):
            out[self.rows(e)] = d[self.rows(e)] @ w[e]
            ab[self.rows(e)] = np.abs(d[self.rows(e)]) @ np.abs(w[e])
        return out, ab

    def weight_grad(self):
        d, x = _f64(self.dout), self.x_rows()
        out = np.stack([d[self.rows(e)].T @ x[self.rows(e)] for e in range(len(self.counts))])
        ab = np.stack([np.abs(d[self.rows(e)]).T @ np.abs(x[self.rows(e)]) for e in range(len(self.counts))])
        return out, ab


def _marked(shape, dtype):
    return torch.full(shape, MARK, dtype=dtype, device=DEV)


def _all(c, out_dtype):
    out = B.grouped_linear(c.x, c.w, c.offsets, row_index=c.index, out=_marked((c.R, c.N), out_dtype))
    dx = B.grouped_input_grad(c.dout, c.w, c.offsets, dx=_marked((c.R, c.K), out_dtype))
    dw = B.grouped_weight_grad(c.dout, c.x, c.offsets, row_index=c.index,
                               dweight=_marked((len(c.counts), c.N, c.K), out_dtype))
    return out, dx, dw


def _check_all(c, out_dtype):
    out, dx, dw = _all(c, out_dtype)
    torch.cuda.synchronize()
    _close("out", out, *c.forward(), c.K, out_dtype)
    _close("dx", dx, *c.input_grad(), c.N, out_dtype)
    _close("dweight", dw, *c.weight_grad(), max(list(c.counts) + [1]), out_dtype)
    return out, dx, dw


COUNTS = {
    "one_row": [1],
    "no_rows_in_any": [0, 0, 0],
    "empty_ends": [0, 3, 0, 17, 0],
    "around_16": [15, 16, 17, 1, 31, 33],
    "around_256": [255, 256, 257, 1],
    "one_has_all": [0] * 5 + [700] + [0] * 6,
    "uneven": [300, 2, 61, 0, 129, 64, 5],
}
WIDTHS = [(8, 8), (64, 64), (72, 264), (200, 136), (520, 40), (256, 512)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("widths", WIDTHS, ids=lambda w: f"{w[0]}x{w[1]}")
@pytest.mark.parametrize("counts", list(COUNTS))
def test_products(counts, widths, dtype):
    c = Case(COUNTS[counts], *widths, dtype, room=3, tokens=50 if counts != "around_16" else None)
    _say(f"[grouped] {counts} {widths} {dtype}")
    _check_all(c, F32 if widths[0] == 72 else dtype)


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F32, BF16)], ids=["bf16_to_f32", "f32_to_bf16"])
def test_result_type_differs(dtype, out_dtype):
    _check_all(Case([40, 0, 300], 136, 72, dtype, first=2, room=5), out_dtype)


def test_most_groups():
    """512 groups, some empty, averages on both sides of the tile choice."""
    g = np.random.default_rng(5)
    _check_all(Case(g.integers(0, 4, 512).tolist(), 64, 40, BF16, tokens=333), BF16)
    _check_all(Case((g.integers(0, 2, 512) * g.integers(0, 220, 512)).tolist(), 40, 24, BF16, first=1), F32)


def test_weight_bound_long_k():
    """K of many stages, few rows (streamed weights) and many."""
    _check_all(Case([1, 2, 0, 5], 2040, 776, BF16), BF16)
    _check_all(Case([130, 60], 2040, 520, BF16), BF16)


LARGE = {
    # (counts, K, N): past one 256 x 256 tile a CU, so that the tiles of the
    # larger products run, with few rows an expert, many, and both sides of the
    # weight gradients' row counts
    "streamed_ragged": ([3, 0, 17, 48, 1, 33, 16, 20] * 8, 1032, 2056),
    "around_256": ([255, 256, 257, 1, 0, 511, 513, 70] * 4, 520, 2056),
    "many_rows": ([1100, 900, 0, 1300, 1000, 1, 1500, 2000], 1032, 1544),
    "narrow_output": ([300, 270] * 100, 72, 264),
    "one_has_all": ([0] * 30 + [5000] + [0] * 33, 264, 2568),
}


@pytest.mark.parametrize("case", list(LARGE))
def test_large_tiles(case):
    counts, K, N = LARGE[case]
    c = Case(counts, K, N, BF16, first=1, room=2, tokens=777, seed=4)
    _say(f"[grouped] large {case}")
    dims = B.make_grouped_dims(c.R, 777, len(counts), K, N, BF16)
    assert B.grouped_workspace_size(dims) > 0 and B.grouped_weight_grad_workspace_size(dims) > 0
    _check_all(c, BF16)
    dw = B.grouped_weight_grad(c.dout, c.x, c.offsets, row_index=c.index)
    dx = B.grouped_input_grad(c.dout, c.w, c.offsets, dx=_marked((c.R, K), F32))
    torch.cuda.synchronize()
    _close("dweight fp32", dw, *c.weight_grad(), max(counts), F32)
    _close("dx fp32", dx, *c.input_grad(), N, F32)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_values_on_large_tiles(value):
    """As above, on the tiles of the larger products: a row's and a K tail's neighbours stay finite."""
    counts = [255, 256, 257, 1, 0, 511, 513, 70] * 4
    c = Case(counts, 520, 2056, BF16, room=2)
    base = (*_all(c, F32)[:2], B.grouped_weight_grad(c.dout, c.x, c.offsets))
    r = 255 + 256 + 256          # the last row of the third group
    x, d = c.x.clone(), c.dout.clone()
    x[r, 519] = value
    d[r, 2055] = value
    out = B.grouped_linear(x, c.w, c.offsets, out=_marked((c.R, c.N), F32))
    dx = B.grouped_input_grad(d, c.w, c.offsets, dx=_marked((c.R, c.K), F32))
    dw = B.grouped_weight_grad(c.dout, x, c.offsets)
    torch.cuda.synchronize()
    keep = torch.ones(c.R, dtype=torch.bool, device=DEV)
    keep[r] = False
    for got, ref in ((out, base[0]), (dx, base[1])):
        assert not torch.isfinite(got[r]).any() and torch.equal(got[keep], ref[keep])
    assert not torch.isfinite(dw[2, :, 519]).any()
    dw[2, :, 519] = base[2][2, :, 519]
    assert torch.equal(dw, base[2])


def test_large_tiles_in_graphs_that_share_a_workspace():
    """The plan and the tile counters live in the workspace: two captured graphs
    and eager calls take turns with one."""
    a = Case([300, 270] * 40, 264, 1032, BF16, tokens=400, seed=6)
    b = Case([3, 0, 17, 48] * 16, 1032, 2056, BF16, seed=7)
    need = 0
    for c in (a, b):
        dims = B.make_grouped_dims(c.R, c.x.shape[0], len(c.counts), c.K, c.N, BF16)
        need = max(need, B.grouped_workspace_size(dims), B.grouped_weight_grad_workspace_size(dims))
    ws = torch.full((need,), 0x7F, dtype=torch.uint8, device=DEV)
    sets = []
    for c in (a, b):
        bufs = (_marked((c.R, c.N), BF16), _marked((c.R, c.K), BF16), _marked((len(c.counts), c.N, c.K), BF16))

        def step(c=c, bufs=bufs):
            B.grouped_linear(c.x, c.w, c.offsets, row_index=c.index, out=bufs[0], workspace=ws)
            B.grouped_input_grad(c.dout, c.w, c.offsets, dx=bufs[1], workspace=ws)
            B.grouped_weight_grad(c.dout, c.x, c.offsets, row_index=c.index, dweight=bufs[2], workspace=ws)

        ref = (B.grouped_linear(c.x, c.w, c.offsets, row_index=c.index),
               B.grouped_input_grad(c.dout, c.w, c.offsets),
               B.grouped_weight_grad(c.dout, c.x, c.offsets, row_index=c.index, weight_grad_dtype=BF16))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        sets.append((g, bufs, ref, step))
    for turn in range(3):
        for g, bufs, ref, step in sets:
            for eager in (False, True):
                for t in bufs:
                    t.fill_(MARK)
                step() if eager else g.replay()
                torch.cuda.synchronize()
                for got, want in zip(bufs, ref):
                    assert torch.equal(got, want), f"turn {turn}"


def test_same_x_row_many_times():
    c = Case([30, 200, 7], 128, 72, BF16, tokens=9)
    c.index.zero_()
    _check_all(c, BF16)


def test_rows_of_nothing():
    x, w = _rand((0, 64), BF16, 1), _rand((3, 40, 64), BF16, 2)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert B.grouped_linear(x, w, off).shape == (0, 40)
    assert B.grouped_input_grad(_rand((0, 40), BF16, 3), w, off).shape == (0, 64)
    dw = B.grouped_weight_grad(_rand((0, 40), BF16, 3), x, off, dweight=_marked((3, 40, 64), F32))
    assert torch.equal(dw, torch.zeros_like(dw))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_stay_in_their_rows(value, dtype):
    """One non-finite element reaches exactly the sums that hold it: no other
    row, no other group, and not through a tile's padding."""
    c = Case([5, 0, 70, 260], 72, 40, dtype, room=2)
    base = _all(c, F32)
    for r in (4, 74, 75 + 259):   # each group's last row
        x, d = c.x.clone(), c.dout.clone()
        x[r, 71] = value
        d[r, 39] = value
        out = B.grouped_linear(x, c.w, c.offsets, out=_marked((c.R, c.N), F32))
        dx = B.grouped_input_grad(d, c.w, c.offsets, dx=_marked((c.R, c.K), F32))
        dw = B.grouped_weight_grad(c.dout, x, c.offsets, weight_grad_dtype=F32)
        torch.cuda.synchronize()
        e = [i for i in range(4) if c.ends[i] <= r < c.ends[i + 1]][0]
        for got, ref in ((out, base[0]), (dx, base[1])):
            assert not torch.isfinite(got[r]).any()
            keep = torch.ones(c.R, dtype=torch.bool, device=DEV)
            keep[r] = False
            assert torch.equal(got[keep], ref[keep])
        assert not torch.isfinite(dw[e, :, 71]).any()
        if np.isinf(value):
            assert torch.equal(out[r], torch.sign(c.w[e, :, 71].float()) * value)
            assert torch.equal(dw[e, :, 71], torch.sign(c.dout[r].float()) * value)
        dw[e, :, 71] = base[2][e, :, 71]
        assert torch.equal(dw, base[2])


def test_bf16_result_keeps_nan():
    c = Case([3], 16, 16, BF16)
    c.x[1, 3] = float("nan")
    out = B.grouped_linear(c.x, c.w, c.offsets)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all()


def test_bad_offsets_and_indexes_stay_in_bounds():
    """Offsets that decrease or pass the rows are clamped, indexes too: the
    values are those of the clamped arguments."""
    c = Case([10, 20, 30, 40], 64, 40, BF16, tokens=50)
    bad = torch.tensor([-5, 30, 12, 1 << 30, -(1 << 30)], dtype=torch.int32, device=DEV)
    good = torch.tensor([0, 30, 30, 100, 100], dtype=torch.int32, device=DEV)
    for args in ((c.x, c.w),):
        a = B.grouped_linear(*args, bad, row_index=c.index, out=_marked((c.R, c.N), BF16))
        b = B.grouped_linear(*args, good, row_index=c.index, out=_marked((c.R, c.N), BF16))
        assert torch.equal(a, b)
    a = B.grouped_input_grad(c.dout, c.w, bad, dx=_marked((c.R, c.K), BF16))
    b = B.grouped_input_grad(c.dout, c.w, good, dx=_marked((c.R, c.K), BF16))
    assert torch.equal(a, b)
    wild = c.index.clone()
    wild[3], wild[50] = -7, 1 << 30
    tame = c.index.clone()
    tame[3], tame[50] = 0, 49
    assert torch.equal(B.grouped_linear(c.x, c.w, c.offsets, row_index=wild),
                       B.grouped_linear(c.x, c.w, c.offsets, row_index=tame))
    assert torch.equal(B.grouped_weight_grad(c.dout, c.x, bad, row_index=wild),
                       B.grouped_weight_grad(c.dout, c.x, good, row_index=tame))


def test_gradients_against_differences():
    """<dout, f> changes with x and W as the gradients say: central differences
    of the 64-bit product are exact up to rounding (f is linear in each), so
    the bound is that of the gradients themselves."""
    c = Case([4, 0, 9], 24, 16, F32, tokens=6)
    dxr = _f64(B.grouped_input_grad(c.dout, c.w, c.offsets))
    dw = _f64(B.grouped_weight_grad(c.dout, c.x, c.offsets, row_index=c.index))
    dx = np.zeros((6, 24))
    np.add.at(dx, c.index.cpu().numpy(), dxr)
    x0, w0, d, idx = _f64(c.x), _f64(c.w), _f64(c.dout), c.index.cpu().numpy()

    def value(x, w):
        return sum(float((d[c.rows(e)] * (x[idx][c.rows(e)] @ w[e].T)).sum()) for e in range(3))

    g = np.random.default_rng(3)
    for _ in range(12):
        vx, vw = g.standard_normal(x0.shape), g.standard_normal(w0.shape)
        num = (value(x0 + vx, w0) - value(x0 - vx, w0)) / 2
        assert abs(num - (dx * vx).sum()) <= 64 * 2.0 ** -24 * (np.abs(dx) * np.abs(vx)).sum() * 10
        num = (value(x0, w0 + vw) - value(x0, w0 - vw)) / 2
        assert abs(num - (dw * vw).sum()) <= 64 * 2.0 ** -24 * (np.abs(dw) * np.abs(vw)).sum() * 10


def test_repeatable_on_side_streams_and_with_a_stale_workspace():
    c = Case([300, 2, 61, 0, 129], 200, 136, BF16, tokens=77)
    ref = _all(c, BF16)
    torch.cuda.synchronize()
    dims = B.make_grouped_dims(c.R, 77, 5, 200, 136, BF16)
    ws = torch.full((max(B.grouped_workspace_size(dims), B.grouped_weight_grad_workspace_size(dims)),), 0xA5,
                    dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s):
            out = B.grouped_linear(c.x, c.w, c.offsets, row_index=c.index, workspace=ws)
            dx = B.grouped_input_grad(c.dout, c.w, c.offsets, workspace=ws)
            dw = B.grouped_weight_grad(c.dout, c.x, c.offsets, row_index=c.index, workspace=ws, weight_grad_dtype=BF16)
        s.synchronize()
        for a, b in zip((out, dx, dw), ref):
            assert torch.equal(a, b)


def test_two_graphs_that_share_a_workspace():
    """Captured, replayed in turn with eager calls between, and with offsets
    that change between the replays."""
    a, b = Case([30, 0, 400], 136, 72, BF16, tokens=40), Case([3, 5, 1], 72, 264, BF16)
    dims = [B.make_grouped_dims(c.R, c.x.shape[0], 3, c.K, c.N, BF16) for c in (a, b)]
    ws = torch.empty(max([B.grouped_workspace_size(d) for d in dims] +
                         [B.grouped_weight_grad_workspace_size(d) for d in dims]), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for c in (a, b):
        bufs = (_marked((c.R, c.N), BF16), _marked((c.R, c.K), BF16), _marked((3, c.N, c.K), F32))

        def step(c=c, bufs=bufs):
            B.grouped_linear(c.x, c.w, c.offsets, row_index=c.index, out=bufs[0], workspace=ws)
            B.grouped_input_grad(c.dout, c.w, c.offsets, dx=bufs[1], workspace=ws)
            B.grouped_weight_grad(c.dout, c.x, c.offsets, row_index=c.index, dweight=bufs[2], workspace=ws)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        torch.cuda.synchronize()
        graphs.append(g)
        outs.append(bufs)
    moved = [torch.tensor([0, 100, 300, 430], dtype=torch.int32, device=DEV),
             torch.tensor([0, 0, 9, 9], dtype=torch.int32, device=DEV)]
    for turn in range(4):
        for c, g, bufs, other in zip((a, b), graphs, outs, moved):
            if turn == 2:
                c.offsets.copy_(other)
            for t in bufs:
                t.fill_(MARK)
            g.replay()
            torch.cuda.synchronize()
            ref = (B.grouped_linear(c.x, c.w, c.offsets, row_index=c.index, out=_marked((c.R, c.N), BF16)),
                   B.grouped_input_grad(c.dout, c.w, c.offsets, dx=_marked((c.R, c.K), BF16)),
                   B.grouped_weight_grad(c.dout, c.x, c.offsets, row_index=c.index))
            torch.cuda.synchronize()
            for got, want in zip(bufs, ref):
                assert torch.equal(got, want), f"turn {turn}"


def test_row_offsets_past_32_bits():
    """x rows whose byte offset passes 2^32 and output elements past 2^31."""
    K, N, tokens = 8, 4096, (1 << 29) + 64       # x: 2^29 rows of 16 bytes
    x = torch.zeros((tokens, K), dtype=BF16, device=DEV)
    R = (1 << 19) + 40                            # out: 2^31 elements and some
    index = torch.zeros(R, dtype=torch.int32, device=DEV)
    index[-1] = tokens - 1
    index[-2] = (1 << 28) + 5
    x[tokens - 1] = 1.0
    x[(1 << 28) + 5] = 2.0
    w = _rand((2, N, K), BF16, 5)
    off = torch.tensor([0, R - 1, R], dtype=torch.int32, device=DEV)
    out = B.grouped_linear(x, w, off, row_index=index)
    s = w.float().sum(2)
    torch.cuda.synchronize()
    bound = 2.0 ** -8 * s.abs() * 2 + 2.0 ** -18
    assert bool(((out[-1].float() - s[1]).abs() <= bound[1]).all())
    assert bool(((out[-2].float() - 2 * s[0]).abs() <= 2 * bound[0]).all())
    assert int(out[:-2].count_nonzero()) == 0


# (a test below has the name of the one above, which runs under this one)
test_gathered_row_offsets_past_32_bits = test_row_offsets_past_32_bits


def _spots_close(name, got, want, absum, n):
    _close(name, got, want, absum, n, BF16)


def test_row_offsets_past_32_bits():
    """x, out, dout and dx of more than 2^31 values: rows at both ends and around value 2^31, zeros elsewhere."""
    K, N = 4096, 4104
    R = (1 << 31) // K + 500
    edge = (1 << 31) // N - 8                         # before K's own edge at (1 << 31) / K
    spots = [0, edge, (1 << 31) // K - 8, R - 16]
    off = torch.tensor([0, 16, edge + 16, R], dtype=torch.int32, device=DEV)
    live = _rand((64, K), BF16, 31), _rand((64, N), BF16, 32)
    w = _rand((3, N, K), BF16, 33, 0.1)
    x, d = torch.zeros((R, K), dtype=BF16, device=DEV), torch.zeros((R, N), dtype=BF16, device=DEV)
    for n, at in enumerate(spots):
        x[at:at + 16], d[at:at + 16] = live[0][16 * n:16 * n + 16], live[1][16 * n:16 * n + 16]
    _say(f"[grouped] {R} rows of {K} and {N}")
    out = B.grouped_linear(x, w, off)
    dx = B.grouped_input_grad(d, w, off)
    dw = B.grouped_weight_grad(d, x, off)
    torch.cuda.synchronize()
    wf, lx, ld = _f64(w), _f64(live[0]), _f64(live[1])
    want = np.zeros((3, N, K))
    ab = np.zeros((3, N, K))
    for n, at in enumerate(spots):
        r = slice(16 * n, 16 * n + 16)
        e = 0 if at < 16 else 1 if at < edge + 16 else 2
        _spots_close(f"out at {at}", out[at:at + 16], lx[r] @ wf[e].T, np.abs(lx[r]) @ np.abs(wf[e]).T, K)
        _spots_close(f"dx at {at}", dx[at:at + 16], ld[r] @ wf[e], np.abs(ld[r]) @ np.abs(wf[e]), N)
        want[e] += ld[r].T @ lx[r]
        ab[e] += np.abs(ld[r]).T @ np.abs(lx[r])
    _close("dw", dw, want, ab, 32, F32)               # zeros add nothing, and no rounding
    for t in (out, dx):
        keep = torch.ones(R, dtype=torch.bool, device=DEV)
        for at in spots:
            keep[at:at + 16] = False
        assert not bool(t.any(dim=1)[keep].any())


def test_weight_offsets_past_32_bits():
    """Weights and weight gradients of more than 2^32 values, in few-row tiles and in tiles of 256 rows."""
    E, N, K = 512, 1032, 8192
    w = torch.zeros((E, N, K), dtype=BF16, device=DEV)
    used = [0, 255, 511]                              # value 2^31 lies in expert 254, 2^32 in 508
    for n, e in enumerate(used):
        w[e] = _rand((N, K), BF16, 40 + n, 0.1)
    for rows in (2, 70):
        c = np.zeros(E, np.int64)
        c[used] = rows
        c[300] = 60 * E if rows == 70 else 0          # on zero weights: more than 48 rows an expert on average
        ends = np.concatenate([[0], np.cumsum(c)])
        R = int(ends[-1])
        off = torch.tensor(ends, dtype=torch.int32, device=DEV)
        x, d = _rand((R, K), BF16, 50), _rand((R, N), BF16, 51)
        _say(f"[grouped] {E} x {N} x {K} weights, {R} rows")
        out, dx = B.grouped_linear(x, w, off), B.grouped_input_grad(d, w, off)
        dw = B.grouped_weight_grad(d, x, off, weight_grad_dtype=BF16)
        torch.cuda.synchronize()
        for e in used:
            r = slice(int(ends[e]), int(ends[e + 1]))
            xe, de, we = _f64(x[r]), _f64(d[r]), _f64(w[e])
            _spots_close(f"out of {e}", out[r], xe @ we.T, np.abs(xe) @ np.abs(we).T, K)
            _spots_close(f"dx of {e}", dx[r], de @ we, np.abs(de) @ np.abs(we), N)
            _spots_close(f"dw of {e}", dw[e], de.T @ xe, np.abs(de).T @ np.abs(xe), rows)
        assert not bool(dw[509].any()) and not bool(dw[1].any())
        del out, dx, dw

def test_refusals():
    x, w = _rand((10, 64), BF16, 1), _rand((3, 40, 64), BF16, 2)
    off = torch.tensor([0, 3, 3, 10], dtype=torch.int32, device=DEV)
    for bad in (dict(x=x.float()), dict(offsets=off[:3]), dict(offsets=off.long()), dict(x=x[:, :32]),
                dict(x=x.cpu()), dict(out=_marked((10, 48), BF16)), dict(x=x.t().contiguous().t()),
                dict(row_index=torch.zeros(10, dtype=torch.int64, device=DEV)),
                dict(workspace=torch.empty(1 << 20, device=DEV))):
        kw = dict(x=x, weight=w, offsets=off) | bad
        with pytest.raises(ValueError):
            B.grouped_linear(**kw)
    with pytest.raises(B.InklingError) as e:
        B.grouped_linear(_rand((4480, 64), BF16, 3), _rand((64, 1024, 64), BF16, 4),
                         torch.arange(65, dtype=torch.int32, device=DEV) * 70, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == B.INKLING_ERR_WORKSPACE
    with pytest.raises(B.InklingError) as e:
        B.grouped_linear(x[:, :60].contiguous(), w[:, :, :60].contiguous(), off)   # 60 columns: not a multiple of 8
    assert e.value.code == B.INKLING_ERR_UNSUPPORTED
    with pytest.raises(B.InklingError) as e:
        B.grouped_linear(x, w, off, out=x[:, :40].contiguous().view(-1)[:0].new_empty(401)[1:].view(10, 40))
    assert e.value.code == B.INKLING_ERR_INVALID_ARGUMENT   # 2-byte aligned output
    with pytest.raises(ValueError):
        B.grouped_weight_grad(_rand((9, 40), BF16, 3), x, off)
    with pytest.raises(ValueError):
        B.grouped_weight_grad(_rand((10, 40), BF16, 3), x, off, dweight=_marked((3, 40, 64), F32),
                              weight_grad_dtype=BF16)
    with pytest.raises(ValueError):
        B.grouped_input_grad(_rand((10, 48), BF16, 3), w, off)
