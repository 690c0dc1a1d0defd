"""Norms on many rows, in every form that few rows do not reach: results stored
past the caches, and workgroups (with one, four or eight vectors a lane) that walk
several rows, loading the next before the sums of the current one.

Against the formulas in 64 bits (on the GPU, a band of rows at a time), with the
bounds of test_gpu_norm.py: a sum over a row is off by at most 64 2^-24 of the sum
of its terms' magnitudes, rstd by 2^-18 of itself, so
  |dy| <= |w| rstd (M + 2^-17 |x - m|) + 2^-22 (|y| + |b|),  M = 64 2^-24 mean|x|,
  |d dx| <= rstd 2^-17 (|c| + mean|c| + |xh| mean|c xh|),
  |d dw| <= (rows + 16) 2^-24 sum|dy xh|, and db likewise,
and half a step, 2^-8 of the value, for a bf16 result."""
import sys

import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(msg, file=sys.stderr, flush=True)


def _form(R, H, dtype):
    """How the kernels hold a row: (vectors a lane, threads of a workgroup that holds a row or None, ragged end)."""
    v = 8 if dtype == BF16 else 4
    n = -(-H // v)
    nv = 1 if n <= 1024 else 4 if n <= 2048 else 8
    return nv, None if n <= 64 else -(-(-(-n // nv)) // 64) * 64, H % v != 0


def _check(name, got, want, bound, dtype):
    bound = bound + 1e-30
    if dtype == BF16:
        bound = bound + 2.0 ** -8 * want.abs()
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"{name}: worst {float((off / bound).max()):.2f} bounds"


def _run(R, H, dtype, kind):
    g = torch.Generator(device=DEV).manual_seed(R + H)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    layer = kind == "layer"
    x, dy = torch.empty((R, H), dtype=dtype, device=DEV), torch.empty((R, H), dtype=dtype, device=DEV)
    x.copy_(rn(R, H) * 2.0 + 0.3)
    dy.copy_(rn(R, H))
    w, b = 1 + 0.3 * rn(H), 0.2 * rn(H) if layer else None
    out, stats = B.norm_forward(x, w, b, eps=1e-6, kind=kind)
    r = B.norm_backward(dy, x, w, stats, kind=kind, bias=layer)
    torch.cuda.synchronize()
    D = torch.float64
    w64, b64 = w.to(D), b.to(D) if layer else torch.zeros((H,), dtype=D, device=DEV)
    sums = [torch.zeros((H,), dtype=D, device=DEV) for _ in range(4)]
    band = max(1, (1 << 24) // H)
    for i in range(0, R, band):
        rows = slice(i, min(R, i + band))
        x64, d64 = x[rows].to(D), dy[rows].to(D)
        m = x64.mean(1, keepdim=True) if layer else torch.zeros_like(x64[:, :1])
        rs = 1.0 / torch.sqrt(((x64 - m) ** 2).mean(1, keepdim=True) + 1e-6)
        y = (x64 - m) * rs * w64 + b64
        M = 64 * 2.0 ** -24 * x64.abs().mean(1, keepdim=True) if layer else torch.zeros_like(m)
        _check(f"out from row {i}", out[rows], y,
               w64.abs() * rs * (M + 2.0 ** -17 * (x64 - m).abs()) + 2.0 ** -22 * (y.abs() + b64.abs()), dtype)
        st = stats[rows].to(D)
        assert bool(((st[:, :1] - m).abs() <= M + 1e-30).all())
        assert bool(((st[:, 1:] - rs).abs() <= 2.0 ** -18 * rs + rs ** 3 * M ** 2).all())
        # the backward takes the stats that it is given
        m, rs = st[:, :1], st[:, 1:]
        xh = (x64 - m) * rs
        c = d64 * w64
        mc, mcx = c.mean(1, keepdim=True), (c * xh).mean(1, keepdim=True)
        dx = rs * (c - xh * mcx - (mc if layer else 0.0))
        _check(f"dx from row {i}", r["dx"][rows], dx,
               rs * 2.0 ** -17 * (c.abs() + c.abs().mean(1, keepdim=True) +
                                  xh.abs() * (c * xh).abs().mean(1, keepdim=True)), dtype)
        for s, t in zip(sums, (d64 * xh, (d64 * xh).abs(), d64, d64.abs())):
            s += t.sum(0)
    n = (R + 16) * 2.0 ** -24
    _check("dweight", r["dweight"], sums[0], n * sums[1], F32)
    if layer:
        _check("dbias", r["dbias"], sums[2], n * sums[3], F32)


PAST = [  # (rows, columns, type, kind, tensors past 256 MB: 2 forward and backward, 3 the backward alone)
    (8192, 6144, BF16, "layer", 3),
    (8192, 6144, BF16, "rms", 3),
    (11000, 6144, BF16, "layer", 2),
    (6000, 12288, BF16, "layer", 2),
    (6000, 12288, BF16, "rms", 2),
    (3000, 12288, F32, "layer", 2),
    (3000, 12288, F32, "rms", 2),
    (5000, 8192, F32, "layer", 2),
    (9000, 4096, F32, "rms", 2),
    (130001, 512, BF16, "layer", 2),
    (300000, 256, BF16, "rms", 2),
    (600001, 128, F32, "layer", 2),
    (1000000, 64, BF16, "layer", 3),
]


@pytest.mark.parametrize("R,H,dtype,kind,tensors", PAST, ids=lambda v: str(v).replace("torch.", ""))
def test_results_past_the_caches(R, H, dtype, kind, tensors):
    values = R * H * (2 if dtype == BF16 else 4)
    assert not _form(R, H, dtype)[2] and values * tensors > 256e6 and (tensors == 2 or values * 2 <= 256e6)
    _say(f"[norm] past the caches: {R} x {H} {dtype} {kind}")
    _run(R, H, dtype, kind)


SEVERAL = [  # rows held by a workgroup, more of them than workgroups in the launch, results within the caches
    (9000, 1000, BF16, "layer", 1), (9000, 1237, BF16, "layer", 1), (3000, 4096, F32, "rms", 1),
    (2500, 8200, BF16, "layer", 4), (2500, 8200, BF16, "rms", 4), (2500, 9001, BF16, "layer", 4),
    (2500, 4100, F32, "layer", 4), (2500, 5001, F32, "rms", 4), (1500, 12288, F32, "layer", 8),
    (1500, 12288, F32, "rms", 8), (1500, 12287, F32, "layer", 8),
]


@pytest.mark.parametrize("R,H,dtype,kind,nv", SEVERAL, ids=lambda v: str(v).replace("torch.", ""))
def test_several_rows_a_workgroup(R, H, dtype, kind, nv):
    vectors, threads, ragged = _form(R, H, dtype)
    cus = torch.cuda.get_device_properties(DEV).multi_processor_count
    assert vectors == nv and threads is not None and R > cus * (2048 // threads)
    assert ragged or R * H * (2 if dtype == BF16 else 4) * 2 <= 256e6
    _say(f"[norm] several rows a workgroup: {R} x {H} {dtype} {kind}")
    _run(R, H, dtype, kind)
