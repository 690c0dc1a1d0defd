"""Grouped products over some of the rows: the offsets of a rank's own experts
begin and end far inside the rows.  Rows and experts outside hold NaN, results
lie between guard values, and the bits are those of the whole call."""
import sys

import numpy as np
import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
MARK = -777.0
GUARD = 1 << 16


def _say(msg):
    print(msg, file=sys.stderr, flush=True)


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def _guarded(shape, dtype):
    """A result between guard values, and the whole buffer."""
    n = int(np.prod(shape))
    buf = torch.full((GUARD + n + GUARD,), MARK, dtype=dtype, device=DEV)
    return buf[GUARD:GUARD + n].view(shape), buf


def _untouched(buf):
    return bool((buf[:GUARD] == MARK).all()) and bool((buf[-GUARD:] == MARK).all())


K, N = 1544, 2056
COUNTS = [500, 812, 0, 256, 700, 1, 333, 900, 512, 0, 640, 255, 1100, 17, 400, 766]


@pytest.fixture(scope="module")
def data():
    ends = np.concatenate([[0], np.cumsum(COUNTS)])
    R = int(ends[-1])
    return dict(ends=ends, R=R, x=_rand((R, K), BF16, 1), dout=_rand((R, N), BF16, 2),
                w=_rand((len(COUNTS), N, K), BF16, 3, 0.1),
                index=torch.tensor(np.random.default_rng(4).permutation(R), dtype=torch.int32, device=DEV))


SPANS = [(0, 16), (8, 16), (4, 16), (12, 16), (2, 10), (15, 16)]


@pytest.mark.parametrize("gather", [False, True], ids=["", "gathered"])
@pytest.mark.parametrize("wdtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("span", SPANS, ids=lambda s: f"{s[0]}to{s[1]}")
def test_weight_gradients_of_some_experts(data, span, wdtype, gather):
    a, b = span
    _say(f"[spans] weight gradients of experts {a} to {b}, {wdtype}, gathered {gather}")
    off = torch.tensor(data["ends"], dtype=torch.int32, device=DEV)
    x, d, idx = data["x"], data["dout"], data["index"] if gather else None
    dims = B.make_grouped_dims(data["R"], data["R"], b - a, K, N, BF16, wdtype)
    assert B.grouped_weight_grad_workspace_size(dims) > 0            # the large tiles
    whole = B.grouped_weight_grad(d, x, off, row_index=idx, weight_grad_dtype=wdtype)
    lo, hi = int(data["ends"][a]), int(data["ends"][b])
    d2, x2 = d.clone(), x.clone()
    outside = torch.ones(data["R"], dtype=torch.bool, device=DEV)
    outside[lo:hi] = False
    d2[outside] = float("nan")
    x2[data["index"][outside].long() if gather else outside] = float("nan")
    dw, buf = _guarded((b - a, N, K), wdtype)
    B.grouped_weight_grad(d2, x2, off[a:b + 1].contiguous(), row_index=idx, dweight=dw)
    torch.cuda.synchronize()
    assert _untouched(buf)
    assert torch.equal(dw, whole[a:b])


@pytest.mark.parametrize("gather", [False, True], ids=["", "gathered"])
@pytest.mark.parametrize("span", [(8, 16), (2, 10)], ids=lambda s: f"{s[0]}to{s[1]}")
def test_rows_of_some_experts(data, span, gather):
    a, b = span
    _say(f"[spans] rows of experts {a} to {b}, gathered {gather}")
    off = torch.tensor(data["ends"], dtype=torch.int32, device=DEV)
    idx = data["index"] if gather else None
    part = off[a:b + 1].contiguous()
    lo, hi = int(data["ends"][a]), int(data["ends"][b])
    dims = B.make_grouped_dims(data["R"], data["R"], b - a, K, N, BF16)
    assert B.grouped_workspace_size(dims) > 0
    for whole, call, cols in (
            (B.grouped_linear(data["x"], data["w"], off, row_index=idx),
             lambda out: B.grouped_linear(data["x"], data["w"][a:b], part, row_index=idx, out=out), N),
            (B.grouped_input_grad(data["dout"], data["w"], off),
             lambda out: B.grouped_input_grad(data["dout"], data["w"][a:b], part, dx=out), K)):
        out, buf = _guarded((data["R"], cols), BF16)
        call(out)
        torch.cuda.synchronize()
        assert _untouched(buf)
        assert torch.equal(out[lo:hi], whole[lo:hi])
        assert bool((out[:lo] == MARK).all()) and bool((out[hi:] == MARK).all())


@pytest.mark.parametrize("wdtype", [F32, BF16], ids=["f32", "bf16"])
def test_offsets_at_the_end_of_the_rows(data, wdtype):
    """Every group empty behind the last row, offsets past the rows, and all rows with the last expert."""
    R, E = data["R"], 8
    for ends in ([R] * 9, [R + 5] * 9, [2 ** 31 - 1] * 9, [-3] * 9, [R - 1000] * 8 + [R], [R - 1000] + [R] * 8):
        _say(f"[spans] offsets {ends[:2]} .. {ends[-2:]}, {wdtype}")
        off = torch.tensor(ends, dtype=torch.int64).clamp(max=2 ** 31 - 1).to(torch.int32).to(DEV)
        dw, buf = _guarded((E, N, K), wdtype)
        B.grouped_weight_grad(data["dout"], data["x"], off, row_index=data["index"], dweight=dw)
        safe = np.maximum.accumulate(np.clip(np.array(ends, np.int64), 0, R))
        torch.cuda.synchronize()
        assert _untouched(buf)
        for e in range(E):
            n = int(safe[e + 1] - safe[e])
            if n == 0:
                assert not bool(dw[e].any())
            else:
                one = torch.tensor([safe[e], safe[e + 1]], dtype=torch.int32, device=DEV)
                ref = B.grouped_weight_grad(data["dout"], data["x"], one, row_index=data["index"],
                                            weight_grad_dtype=wdtype)
                assert n == 1000 and torch.equal(dw[e], ref[0]) and bool(ref.any())


def test_weight_gradients_of_mostly_empty_experts():
    """Tiles without a K loop in a row: most experts have no rows, and each workgroup takes several of their tiles."""
    E, k, n = 256, 264, 520
    counts = np.zeros(E, np.int64)
    counts[[0, 7, 100, 101, 255]] = [300, 1, 700, 64, 33]
    ends = np.concatenate([[40], 40 + np.cumsum(counts)])
    R = int(ends[-1]) + 9
    dims = B.make_grouped_dims(R, R, E, k, n, BF16, F32)
    assert B.grouped_weight_grad_workspace_size(dims) > 0
    x, d = _rand((R, k), BF16, 5), _rand((R, n), BF16, 6)
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    _say(f"[spans] {E} experts, 5 with rows")
    first = None
    for turn in range(4):
        dw, buf = _guarded((E, n, k), F32)
        B.grouped_weight_grad(d, x, off, dweight=dw)
        torch.cuda.synchronize()
        assert _untouched(buf)
        assert first is None or torch.equal(dw, first), f"turn {turn}"
        first = dw
    full = torch.ones(E, dtype=torch.bool, device=DEV)
    for e in np.flatnonzero(counts):
        r = slice(int(ends[e]), int(ends[e + 1]))
        d64, x64 = d[r].cpu().double(), x[r].cpu().double()
        # products of bf16 are exact in fp32; n sums move by at most 2 n 2^-24 of the magnitudes
        bound = 2 * float(counts[e]) * 2.0 ** -24 * (d64.abs().t() @ x64.abs()) + 1e-30
        assert bool(((first[e].cpu().double() - d64.t() @ x64).abs() <= bound).all()), e
        full[e] = False
    assert not bool(first[full].any())


@pytest.fixture(scope="module")
def far_rows():
    """x of 2^29 + 64 rows of 16 bytes, and 40 of its rows on both sides of bytes 2^31, 2^32 and 2^33."""
    x = torch.zeros(((1 << 29) + 64, 8), dtype=BF16, device=DEV)
    at = torch.cat([torch.arange(b - 5, b + 5) for b in (1 << 27, 1 << 28, (1 << 29) - 5, (1 << 29) + 59)])
    rows = _rand((40, 8), BF16, 11)
    x[at.to(DEV)] = rows
    return x, at, rows


@pytest.mark.parametrize("E,R,n", [(2, 300, 40), (2, 5000, 4096), (512, 1000, 40960)],
                         ids=["small_tiles", "large_tiles", "streamed_weights"])
def test_gathered_rows_past_32_bits(far_rows, E, R, n):
    """Rows of x whose byte offsets pass 2^32, against the same rows of a short x."""
    x, at, rows = far_rows
    near = torch.tensor(np.random.default_rng(R).integers(0, 40, R), dtype=torch.int32)
    far = at[near.long()].to(torch.int32).to(DEV)
    near = near.to(DEV)
    ends = np.sort(np.random.default_rng(E).integers(0, R + 1, E + 1))
    ends[0], ends[-1] = 0, R
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    w, d = _rand((E, n, 8), BF16, 12), _rand((R, n), BF16, 13)
    _say(f"[spans] gathered rows past 2^32 bytes, {E} experts, {R} rows, {n} columns")
    out, want = B.grouped_linear(x, w, off, row_index=far), B.grouped_linear(rows, w, off, row_index=near)
    dw, dwant = (B.grouped_weight_grad(d, x, off, row_index=far),
                 B.grouped_weight_grad(d, rows, off, row_index=near))
    torch.cuda.synchronize()
    assert bool(want.any()) and torch.equal(out, want)
    assert bool(dwant.any()) and torch.equal(dw, dwant)


def _step(data, off, w, bufs, ws=None, wws=None):
    B.grouped_linear(data["x"], w, off, row_index=data["index"], out=bufs[0], workspace=ws)
    B.grouped_input_grad(data["dout"], w, off, dx=bufs[1], workspace=ws)
    B.grouped_weight_grad(data["dout"], data["x"], off, row_index=data["index"], dweight=bufs[2], workspace=wws)


def _bufs(data, E):
    return [torch.full(s, MARK, dtype=BF16, device=DEV) for s in ((data["R"], N), (data["R"], K), (E, N, K))]


def test_a_graph_whose_offsets_move(data):
    """Captured with the later experts' offsets, replayed with others in the same memory: late, early, all at the
    end, none; each replay against eager calls of the same offsets."""
    E, ends, R = 8, data["ends"], data["R"]
    off = torch.tensor(ends[8:], dtype=torch.int32, device=DEV)
    w, bufs = data["w"][:E], _bufs(data, E)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(data, off, w, bufs)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _step(data, off, w, bufs)
    for moved in (ends[8:], ends[:9], [R - 2500] * 8 + [R], [R] * 9, ends[4:13], [R // 2] * 4 + [R] * 5):
        off.copy_(torch.tensor(np.asarray(moved), dtype=torch.int32))
        for t in bufs:
            t.fill_(MARK)
        g.replay()
        torch.cuda.synchronize()
        want = _bufs(data, E)
        _step(data, off, w, want)
        torch.cuda.synchronize()
        for a, b in zip(bufs, want):
            assert torch.equal(a, b), list(moved)[:3]


def test_two_calls_at_once(data):
    """Two streams, each with workspaces of its own, over the two halves of the experts."""
    off = torch.tensor(data["ends"], dtype=torch.int32, device=DEV)
    halves = [(off[:9].contiguous(), data["w"][:8]), (off[8:].contiguous(), data["w"][8:])]
    want = [_bufs(data, 8) for _ in halves]
    for (o, w), b in zip(halves, want):
        _step(data, o, w, b)
    torch.cuda.synchronize()
    dims = B.make_grouped_dims(data["R"], data["R"], 8, K, N, BF16)
    streams = [torch.cuda.Stream() for _ in halves]
    got = [_bufs(data, 8) for _ in halves]
    spaces = [[torch.empty(n, dtype=torch.uint8, device=DEV) for n in
               (B.grouped_workspace_size(dims), B.grouped_weight_grad_workspace_size(dims))] for _ in halves]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, (o, w), b, (ws, wws) in zip(streams, halves, got, spaces):
            with torch.cuda.stream(st):
                _step(data, o, w, b, ws, wws)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for t, u in zip(a, b):
            assert torch.equal(t, u)
