"""The 8-bit checkpoint's stated error on blocks of values near fp32's smallest,
the sigmoid where its exponential passes fp32, and data past the caches."""
import numpy as np
import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _values(ck, R, I):
    """What the checkpoint's bytes stand for, [R, 2 I] in 64 bits."""
    raw = ck.cpu().numpy()
    q = raw[:R * 2 * I].view(np.int8).reshape(R, 2 * I).astype(np.float64)
    e = raw[R * 2 * I:].reshape(R, I // 16).astype(np.float64) - 127
    return q * np.repeat(np.exp2(e), 32, axis=1)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_error_of_kept_values_down_to_the_smallest(dtype):
    """Blocks whose largest value goes from the smallest subnormal past 127 2^-127: off by at most the larger of
    max|h| / 127 and 2^-127, and the latter is needed: max|h| / 127 alone does not hold where e is -126."""
    g = torch.Generator().manual_seed(3)
    tops = 2.0 ** torch.arange(-149, -108, dtype=torch.float64)
    tops = torch.cat([tops, 1.75 * tops, torch.tensor([127 * 2.0 ** -127, 128 * 2.0 ** -127], dtype=torch.float64)])
    h = (torch.rand((len(tops), 32), generator=g, dtype=torch.float64) * 2 - 1) * tops[:, None]
    h[:, 7] = tops
    h = h.to(dtype)
    _, ck = B.swiglu_forward(h.to(DEV))
    torch.cuda.synchronize()
    h = h.double().numpy()
    off, top = np.abs(_values(ck, len(tops), 16) - h).max(1), np.abs(h).max(1)
    assert (off <= np.maximum(top / 127, 2.0 ** -127)).all()
    assert (off[top > 127 * 2.0 ** -127] <= top[top > 127 * 2.0 ** -127] / 127).all()
    assert (off > top / 127).any()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_gates_below_the_exponentials_range(dtype):
    """exp(-g) passes fp32 below -88.7; where the sigmoid is less than 2^-126 it may come out as 0, and act is off by
    at most |g u| 2^-126 and its own rounding."""
    gates = torch.tensor([-80.0, -87.0, -88.0, -88.5, -89.0, -90.0, -95.0, -100.0, -103.0, -104.0, -110.0, -200.0,
                          -1e4, -1e20, -1e30, -3e38])
    h = torch.zeros((1, 32))
    h[0, 0::2], h[0, 1::2] = gates, 1.5
    h = h.to(dtype)
    act, _ = B.swiglu_forward(h.to(DEV))
    torch.cuda.synchronize()
    g = h[0, 0::2].double().numpy()
    with np.errstate(over="ignore"):
        s = np.where(g < -700, 0.0, 1.0 / (1.0 + np.exp(-np.maximum(g, -700))))
    want = g * s * 1.5
    rel = (1.5 * np.minimum(np.abs(g), 128.0) + 16.0) * 2.0 ** -24 + (2.0 ** -8 if dtype == BF16 else 0.0)
    bound = np.abs(want) * rel + np.where(g < -87.3, np.abs(g) * 1.5 * 2.0 ** -126, 0.0)
    assert (np.abs(act[0].cpu().double().numpy() - want) <= bound).all()


@pytest.mark.parametrize("dtype,R,I", [(BF16, 32011, 1024), (F32, 20011, 1024), (BF16, 200003, 208), (F32, 400009, 48)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_data_past_the_caches(dtype, R, I):
    """More than 256 MB takes kernels that store past the caches: the bits are those of short calls on bands of the
    rows, which do not, and rows from the count on are left as they were."""
    es = 2 if dtype == BF16 else 4
    assert R * I * (2 + 3 * es) > 256e6 and 1000 * I * (2 + 4 * es) < 256e6
    g = torch.Generator(device=DEV).manual_seed(R)
    h = (torch.randn((R, 2 * I), generator=g, device=DEV) * 2).to(dtype)
    da = torch.randn((R, I), generator=g, device=DEV).to(dtype)
    gamma = torch.rand((R,), generator=g, device=DEV)
    used = R - 77
    n = torch.tensor([used], dtype=torch.int32, device=DEV)
    bufs = [torch.full((R, w), -777.0, dtype=dtype, device=DEV) for w in (I, 2 * I, I)]
    dgamma = torch.full((R,), -777.0, device=DEV)
    act, ck = B.swiglu_forward(h, gamma, row_count=n, out=bufs[0])
    r = B.swiglu_backward(da, ck, gamma, row_count=n, dh=bufs[1], act=bufs[2], dgamma=dgamma)
    for i in (0, 1000, R // 2, used - 1000):
        rows = slice(i, i + 1000)
        want, ck2 = B.swiglu_forward(h[rows], gamma[rows])
        r2 = B.swiglu_backward(da[rows], ck2, gamma[rows])
        torch.cuda.synchronize()
        assert torch.equal(act[rows], want), i
        assert torch.equal(ck[i * 2 * I:(i + 1000) * 2 * I], ck2[:1000 * 2 * I]), i
        at = R * 2 * I + i * (I // 16)
        assert torch.equal(ck[at:at + 1000 * (I // 16)], ck2[1000 * 2 * I:]), i
        for k in ("dh", "act", "dgamma"):
            assert torch.equal(r[k][rows], r2[k]), (k, i)
    for t in (*bufs, dgamma):
        assert bool((t[used:] == -777.0).all()) and not bool((t[:used] == -777.0).any())
