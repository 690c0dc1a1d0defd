"""Norm rows at the edges of fp32 and of the kernels' forms: every way a row is
held (lanes of a wave, a workgroup with one, four or eight vectors a lane), whole
vectors and a ragged end, lanes left over behind the row."""
import sys

import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(msg, file=sys.stderr, flush=True)


def _vec(H, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((H,), generator=g) * scale + shift).to(DEV)


# lanes without columns follow the row in all of them
FORMS = [(20, BF16), (77, BF16), (136, BF16), (300, F32), (1000, BF16), (1001, BF16), (1237, F32), (8200, BF16),
         (9001, BF16), (4100, F32), (5001, F32), (8200, F32), (8201, F32)]


@pytest.mark.parametrize("H,dtype", FORMS, ids=lambda v: str(v).replace("torch.", ""))
def test_constant_rows_of_large_values(H, dtype):
    """x = 2^113 and eps = 2^-40: (0 - mean) rstd would pass fp32, while every x - mean is 0.

    n 2^113 is exact for n < 2^24, so the mean is exact, x - mean is 0 and out the bias; rstd is 2^20 exactly.
    dx = rstd (c - mean c) with c = dout w: one rounding a product, a mean off by 64 2^-24 mean|c| at most (32
    values one after another and 22 levels of a tree, and the quotient), two more roundings, and dx's own."""
    _say(f"[norm] constant rows, {H} {dtype}")
    x = torch.full((3, H), 2.0 ** 113, device=DEV).to(dtype)
    w, b = _vec(H, 1, 0.3, 1.0), _vec(H, 2)
    dy = torch.stack([_vec(H, 3 + i) for i in range(3)]).to(dtype)
    out, stats = B.norm_forward(x, w, b, eps=2.0 ** -40)
    r = B.norm_backward(dy, x, w, stats, bias=True)
    torch.cuda.synchronize()
    assert torch.equal(stats.cpu(), torch.tensor([[2.0 ** 113, 2.0 ** 20]] * 3))
    assert torch.equal(out, b.to(dtype).expand(3, H))
    c = dy.cpu().double() * w.cpu().double()
    want = 2.0 ** 20 * (c - c.mean(1, keepdim=True))
    bound = 2.0 ** 20 * (67 * 2.0 ** -24 * c.abs().mean(1, keepdim=True) + 3 * 2.0 ** -24 * c.abs())
    bound = bound + (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * want.abs()
    assert bool(((r["dx"].cpu().double() - want).abs() <= bound).all())
    assert not bool(r["dweight"].any())
    assert bool(torch.isfinite(r["dbias"]).all()) and bool(r["dbias"].any())


F32_WIDTHS = [20, 77, 300, 1000, 1237, 4100, 5001, 8200, 8201, 16383]


@pytest.mark.parametrize("H", F32_WIDTHS)
def test_constant_rows_whose_sum_is_rounded(H):
    """A row of one fp32 value, far from 0, is its mean whatever its long sum was rounded to.

    The first mean is off by d <= 64 2^-24 |x|; x - mean is exact (values within a factor of two) and the same c,
    |c| <= d, in every column; the mean of those is c to 66 2^-24 of itself.  So out is off by at most
    |w| rstd 66 2^-24 d and two roundings of the sum with the bias; the mean that is kept, by its own rounding."""
    value = torch.tensor([10000.333, 0.1, -33333.33, 12345.678, 1e-3], dtype=F32)
    x = value[:, None].expand(-1, H).contiguous().to(DEV)
    w, b = _vec(H, 1, 0.3, 1.0), _vec(H, 2)
    out, stats = B.norm_forward(x, w, b, eps=1e-6)
    torch.cuda.synchronize()
    v, w, b = value.double()[:, None], w.cpu().double(), b.cpu().double()
    d = 64 * 2.0 ** -24 * v.abs()
    _say(f"[norm] constant rows, {H}: out off by {float((out.cpu().double() - b).abs().max()):.2e}")
    assert bool(((out.cpu().double() - b).abs() <= w.abs() * 1e3 * 66 * 2.0 ** -24 * d + 2.0 ** -23 * b.abs()).all())
    assert bool(((stats.cpu().double()[:, :1] - v).abs() <= 2.0 ** -24 * v.abs() + 66 * 2.0 ** -24 * d).all())


@pytest.mark.parametrize("H", F32_WIDTHS)
def test_small_spread_about_a_large_mean(H):
    """mean 10000, spread 0.01 (ten steps of fp32 there), against 64 bits.

    With d as above and e the mean of |x - mean| plus d: x - mean is exact, its mean off by 64 2^-24 e; the
    variance by 2^-18 of itself and of d^2, rstd by as much of itself (half, and a few roundings)."""
    g = torch.Generator().manual_seed(H)
    x = (torch.randn((4, H), generator=g) * 0.01 + 10000.0).to(F32)
    w, b = _vec(H, 1, 0.3, 1.0), _vec(H, 2)
    out, stats = B.norm_forward(x.to(DEV), w, b, eps=1e-6)
    torch.cuda.synchronize()
    x, w, b = x.double(), w.cpu().double(), b.cpu().double()
    m = x.mean(1, keepdim=True)
    var = ((x - m) ** 2).mean(1, keepdim=True)
    r = 1.0 / torch.sqrt(var + 1e-6)
    y = (x - m) * r * w + b
    d = 64 * 2.0 ** -24 * x.abs().mean(1, keepdim=True)
    e = (x - m).abs().mean(1, keepdim=True) + d
    rel = 2.0 ** -18 * (var + d * d) / (var + 1e-6) + 2.0 ** -21
    bound = w.abs() * r * (64 * 2.0 ** -24 * e + rel * ((x - m).abs() + 64 * 2.0 ** -24 * e)) + 2.0 ** -23 * (y.abs() + b.abs())
    off = (out.cpu().double() - y).abs()
    _say(f"[norm] spread 0.01 about 10000, {H}: out off by {float(off.max()):.2e}, {float((off / bound).max()):.2f} bounds")
    assert bool((off <= bound).all())
    assert bool(((stats.cpu().double()[:, :1] - m).abs() <= 2.0 ** -24 * m.abs() + 64 * 2.0 ** -24 * e).all())
    assert bool(((stats.cpu().double()[:, 1:] - r).abs() <= rel * r).all())


@pytest.mark.parametrize("H", [20, 1000, 1237, 6144, 9001, 16384])
def test_bf16_rows_a_few_steps_about_a_large_mean(H):
    """10000 and the bf16 values next to it (steps of 64): sums of at most 2^14 multiples of 64 below 2^9 of them are
    exact, so the mean is off by its quotient's rounding, 2^-24 of itself, and the variance by 2^-18 of itself."""
    g = torch.Generator().manual_seed(H)
    x = (9984.0 + 64.0 * torch.randint(-2, 3, (4, H), generator=g)).to(BF16)
    w, b = _vec(H, 1, 0.3, 1.0), _vec(H, 2)
    out, stats = B.norm_forward(x.to(DEV), w, b, eps=1e-6)
    torch.cuda.synchronize()
    x, w, b = x.double(), w.cpu().double(), b.cpu().double()
    m = x.mean(1, keepdim=True)
    r = 1.0 / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + 1e-6)
    y = (x - m) * r * w + b
    off = 2.0 ** -24 * m.abs()
    bound = w.abs() * r * (off + 2.0 ** -18 * (x - m).abs()) + 2.0 ** -22 * (y.abs() + b.abs()) + 2.0 ** -8 * y.abs()
    assert bool(((out.cpu().double() - y).abs() <= bound).all())
    assert bool(((stats.cpu().double()[:, :1] - m).abs() <= off).all())
