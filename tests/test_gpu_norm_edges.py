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
