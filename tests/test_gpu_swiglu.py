"""SwiGLU with the 8-bit checkpoint against the formulas in 64 bits.

The checkpoint's bytes are compared one by one with the definition.  The other
results follow fp32 arithmetic.  Sigmoid: exp(-g) as 2^(-g log2 e) is off by at
most (1.5 |g| + 2) 2^-24 of itself (the product's rounding and the constant's,
scaled by ln 2 |g| log2 e = |g|; the exponential one step), 1 + exp and the
reciprocal add 3 more; each further product adds one: REL(g) = (1.5 |g| + 16)
2^-24 covers every product of s, g, u, gamma and dact.  In dg the factor
1 + g (1 - s) cancels, so its error is taken against s (1 + |g|) |dp u|, twice.
A bf16 result adds half a step, 2^-8 of the value; results below 1e-30 (where
exp overflows and s is 0) are taken as 0.
"""
import ctypes
import sys

import numpy as np
import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
MARK = -777.0


def _say(msg):
    print(msg, file=sys.stderr, flush=True)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _make(R, I, dtype, seed=1, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn((R, 2 * I), generator=g) * scale
    return (h.to(dtype).to(DEV), torch.rand((R,), generator=g).to(DEV) - 0.3,
            torch.randn((R, I), generator=g).to(dtype).to(DEV))


def _keep(h):
    """Definition of the checkpoint in 64 bits: (int8 [R, 2I], bytes [R, I/16], values that come back)."""
    R, W = h.shape
    b = h.reshape(R, W // 32, 32)
    with np.errstate(invalid="ignore"):
        bad = ~np.isfinite(b).all(2)
    top = np.where(bad, 1.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(2))
    # the smallest e >= -126 with top <= 127 2^e
    e = np.where(top > 0, np.maximum(np.frexp(top)[1] - 8, -126), -126)
    while (top > 127.0 * np.exp2(e)).any():
        e = np.where(top > 127.0 * np.exp2(e), e + 1, e)
    assert ((top > 127.0 * np.exp2(e - 1)) | (e == -126)).all()
    q = np.where(bad[:, :, None], 0.0, np.rint(np.where(bad[:, :, None], 0.0, b) / np.exp2(e)[:, :, None]))
    back = np.where(bad[:, :, None], np.nan, q * np.exp2(e)[:, :, None])
    return q.reshape(R, W).astype(np.int8), np.where(bad, 255, e + 127).astype(np.uint8), back.reshape(R, W)


def _split(ck, R, I):
    raw = ck.cpu().numpy()
    return raw[:R * 2 * I].view(np.int8).reshape(R, 2 * I), raw[R * 2 * I:R * 2 * I + R * I // 16].reshape(R, I // 16)


def _sig(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def _rel(g):
    return (1.5 * np.minimum(np.abs(g), 90.0) + 16.0) * 2.0 ** -24


def _check(name, got, want, bound, dtype):
    got = _f64(got)
    bound = bound + (2.0 ** -8 * np.abs(want) if dtype == BF16 else 0.0) + 1e-30
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{name}: {int(bad.sum())} off, first at {np.argwhere(bad)[:3].tolist()}"


def _check_forward(act, h, gamma, dtype):
    g, u = h[:, 0::2], h[:, 1::2]
    want = gamma * g * _sig(g) * u
    _check("act", act, want, np.abs(want) * _rel(g), dtype)


def _check_backward(r, back, gamma, da, dtype):
    g, u = back[:, 0::2], back[:, 1::2]
    s = _sig(g)
    p = g * s * u
    dp = gamma * da
    _check("act again", r["act"], gamma * p, np.abs(gamma * p) * _rel(g), dtype)
    dg = dp * u * s * (1.0 + g * (1.0 - s))
    du = dp * g * s
    _check("dg", r["dh"][:, 0::2], dg, 2 * np.abs(dp * u) * s * (1.0 + np.abs(g)) * _rel(g), dtype)
    _check("du", r["dh"][:, 1::2], du, np.abs(du) * _rel(g), dtype)
    n = g.shape[1]
    _check("dgamma", r["dgamma"], (da * p).sum(1), (np.abs(da * p) * (_rel(g) + n * 2.0 ** -24)).sum(1), F32)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,I", [(1, 16), (1, 2048), (3, 48), (7, 208), (65, 768), (130, 64), (33, 528), (5, 4096)])
def test_against_64_bits(R, I, dtype):
    _say(f"[swiglu] {R} x {I} {dtype}")
    h, gamma, da = _make(R, I, dtype, seed=R + I, scale=2.0)
    act, ck = B.swiglu_forward(h, gamma)
    r = B.swiglu_backward(da, ck, gamma)
    torch.cuda.synchronize()
    h64, gm = _f64(h), _f64(gamma)[:, None]
    q, e, back = _keep(h64)
    gq, ge = _split(ck, R, I)
    assert np.array_equal(ge, e) and np.array_equal(gq, q)
    assert (np.abs(back - h64).reshape(R, -1, 32).max(2) <= np.abs(h64).reshape(R, -1, 32).max(2) / 127).all()
    _check_forward(act, h64, gm, dtype)
    _check_backward(r, back, gm, _f64(da), dtype)


def test_without_gamma_and_optional_results():
    h, _, da = _make(40, 96, BF16, 3)
    act, ck = B.swiglu_forward(h)
    one = torch.ones(40, device=DEV)
    act1, ck1 = B.swiglu_forward(h, one)
    assert torch.equal(act, act1) and torch.equal(ck, ck1)
    full = B.swiglu_backward(da, ck, one)
    part = B.swiglu_backward(da, ck, want_act=False, want_dgamma=False)
    assert part["act"] is None and part["dgamma"] is None and torch.equal(part["dh"], full["dh"])
    alone, none = B.swiglu_forward(h, save=False)
    assert none is None and torch.equal(alone, act)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_block_scale_edges(dtype):
    """Zeros, powers of two, the carry at 127/64, the type's extremes and subnormals."""
    tops = [0.0, 1.0, 127.0, 127.5, 128.0, 1.984375, 1.9921875, 2.0 ** -126, 2.0 ** -133, 3.0e38, 2.0 ** 127,
            2.0 ** -120 * 1.5, -1.0, -255.0, 63.5, 64.0]
    g = torch.Generator().manual_seed(5)
    h = torch.rand((len(tops), 32), generator=g).double() * 2 - 1
    for i, t in enumerate(tops):
        h[i] = h[i] * abs(t) * 0.99
        h[i, (5 * i) % 32] = t
    h = h.to(dtype)
    act, ck = B.swiglu_forward(h.to(DEV), checkpoint=None)
    torch.cuda.synchronize()
    q, e, _ = _keep(h.double().numpy())
    gq, ge = _split(ck, len(tops), 16)
    assert np.array_equal(ge, e), (ge[:, 0], e[:, 0])
    assert np.array_equal(gq, q)


def test_ties_go_to_the_even_step():
    h = torch.zeros((1, 32))
    h[0, 0] = 64.0                                    # e = 0: steps of 1
    h[0, 1:9] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 3.4999998, 63.5])
    _, ck = B.swiglu_forward(h.to(DEV))
    torch.cuda.synchronize()
    gq, ge = _split(ck, 1, 16)
    assert ge[0, 0] == 127
    assert gq[0, :9].tolist() == [64, 0, 2, 2, 0, -2, -2, 3, 64]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_non_finite_blocks(dtype):
    h, gamma, da = _make(6, 64, dtype, 9)
    for r, v in ((1, float("nan")), (2, float("inf")), (4, -float("inf"))):
        h[r, 40] = v                                  # the second block of its row
    act, ck = B.swiglu_forward(h, gamma)
    r = B.swiglu_backward(da, ck, gamma)
    torch.cuda.synchronize()
    q, e, back = _keep(_f64(h))
    gq, ge = _split(ck, 6, 64)
    assert np.array_equal(ge, e) and np.array_equal(gq, q)
    bad = np.isnan(back)
    assert np.array_equal(np.isnan(_f64(r["dh"])), bad)
    assert np.array_equal(np.isnan(_f64(r["act"])), bad[:, 0::2])
    assert np.array_equal(np.isnan(_f64(r["dgamma"])), bad.any(1))
    # forward: the elements themselves; silu(inf) = inf, silu(-inf) = NaN
    assert np.isnan(_f64(act)[1, 20]) and np.isinf(_f64(act)[2, 20]) and np.isfinite(np.delete(_f64(act), 20, 1)).all()


def test_large_gates():
    """Where exp overflows or vanishes, the limits of the sigmoid."""
    h = torch.zeros((2, 32))
    h[0, 0::2] = torch.tensor([-200.0, -100.0, -89.0, -50.0, -20.0, 0.0, 20.0, 50.0, 89.0, 100.0, 200.0, -1.28, 1.28,
                               -0.0, 1e-20, -1e-20])
    h[:, 1::2] = 2.0
    h[1] = h[0]
    gamma, da = torch.tensor([1.0, -0.5]), torch.ones((2, 16))
    for dtype in (BF16, F32):
        hd, dd = h.to(dtype).to(DEV), da.to(dtype).to(DEV)
        act, ck = B.swiglu_forward(hd, gamma.to(DEV))
        r = B.swiglu_backward(dd, ck, gamma.to(DEV))
        torch.cuda.synchronize()
        gm = gamma.double().numpy()[:, None]
        _check_forward(act, _f64(hd), gm, dtype)
        _check_backward(r, _keep(_f64(hd))[2], gm, _f64(dd), dtype)


@pytest.mark.parametrize("count", [-3, 0, 1, 37, 50, 1000])
def test_row_count(count):
    """Rows from the count on keep what every buffer held; a count out of range is clamped."""
    R, I = 50, 80
    h, gamma, da = _make(R, I, BF16, 11)
    n = torch.tensor([count], dtype=torch.int32, device=DEV)
    size = B.swiglu_checkpoint_size(B.make_swiglu_dims(R, I, BF16))
    ck = torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV)
    out = torch.full((R, I), MARK, dtype=BF16, device=DEV)
    bufs = dict(dh=torch.full((R, 2 * I), MARK, dtype=BF16, device=DEV), act=torch.full((R, I), MARK, dtype=BF16,
                                                                                     device=DEV),
                dgamma=torch.full((R,), MARK, device=DEV))
    B.swiglu_forward(h, gamma, row_count=n, out=out, checkpoint=ck)
    B.swiglu_backward(da, ck, gamma, row_count=n, **bufs)
    act, ck2 = B.swiglu_forward(h, gamma)
    r = B.swiglu_backward(da, ck2, gamma)
    torch.cuda.synchronize()
    k = min(max(count, 0), R)
    for got, want in ((out, act), (bufs["dh"], r["dh"]), (bufs["act"], r["act"]), (bufs["dgamma"], r["dgamma"])):
        assert torch.equal(got[:k], want[:k]) and bool((got[k:] == MARK).all())
    for got, want, w in zip(_split(ck, R, I), _split(ck2, R, I), (np.int8, np.uint8)):
        assert np.array_equal(got[:k], want[:k]) and (got[k:] == 0x5A).all()


def test_gradients_against_differences():
    """Central differences of act at the values that come back: the error of a
    step d is the third derivative, below d^2 |f'''| / 6 with |f'''| < 2 (|u| + 1)."""
    h, gamma, da = _make(4, 32, F32, 13)
    _, ck = B.swiglu_forward(h, gamma)
    r = B.swiglu_backward(da, ck, gamma)
    torch.cuda.synchronize()
    back, gm, d = _keep(_f64(h))[2], _f64(gamma)[:, None], _f64(da)

    def value(b, g):
        return (d * g * b[:, 0::2] * _sig(b[:, 0::2]) * b[:, 1::2]).sum(1)

    step = 1e-4
    dh = _f64(r["dh"])
    for c in range(64):
        up, dn = back.copy(), back.copy()
        up[:, c] += step
        dn[:, c] -= step
        num = (value(up, gm) - value(dn, gm)) / (2 * step)
        room = step ** 2 * (np.abs(d * gm).max(1) * (np.abs(back).max(1) + 1)) + 2e-6 * (1 + np.abs(back).max(1)) ** 2
        assert (np.abs(num - dh[:, c]) <= room).all()
    num = (value(back, gm + step) - value(back, gm - step)) / (2 * step)
    assert np.abs(num - _f64(r["dgamma"])).max() <= 1e-4


def test_captured_in_a_graph_and_on_a_side_stream():
    h, gamma, da = _make(300, 208, BF16, 15)
    n = torch.tensor([300], dtype=torch.int32, device=DEV)
    size = B.swiglu_checkpoint_size(B.make_swiglu_dims(300, 208, BF16))
    ck = torch.zeros((size,), dtype=torch.uint8, device=DEV)
    out = torch.zeros((300, 208), dtype=BF16, device=DEV)
    bufs = dict(dh=torch.zeros((300, 416), dtype=BF16, device=DEV), act=torch.zeros((300, 208), dtype=BF16, device=DEV),
                dgamma=torch.zeros((300,), device=DEV))

    def step():
        B.swiglu_forward(h, gamma, row_count=n, out=out, checkpoint=ck)
        B.swiglu_backward(da, ck, gamma, row_count=n, **bufs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for count in (300, 7, 222):
        n.fill_(count)
        for t in (out, *bufs.values()):
            t.fill_(MARK)
        g.replay()
        torch.cuda.synchronize()
        act, ck2 = B.swiglu_forward(h, gamma)
        r = B.swiglu_backward(da, ck2, gamma)
        torch.cuda.synchronize()
        for got, want in ((out, act), *((bufs[k], r[k]) for k in bufs)):
            assert torch.equal(got[:count], want[:count]) and bool((got[count:] == MARK).all())


def test_byte_offsets_past_32_bits():
    """The last rows of a checkpoint of more than 2^32 bytes, h of more than 2^33."""
    I, R = 4096, (1 << 19) + 100
    h = torch.zeros((R, 2 * I), dtype=BF16, device=DEV)
    tail, gamma, da = _make(64, I, BF16, 21)
    h[-64:] = tail
    act, ck = B.swiglu_forward(h)
    want, ck2 = B.swiglu_forward(tail)
    assert torch.equal(act[-64:], want) and int(act[:-64].count_nonzero()) == 0
    del h, act
    d = torch.zeros((R, I), dtype=BF16, device=DEV)
    d[-64:] = da
    r, r2 = B.swiglu_backward(d, ck), B.swiglu_backward(da, ck2)
    for k in ("dh", "act", "dgamma"):
        assert torch.equal(r[k][-64:], r2[k])
    assert int(r["dh"][:-64].count_nonzero()) == 0


def test_more_rows_than_one_launch_counts():
    """2^30 lanes and beyond: the forward goes over the rows in bands.  Rows at both ends, where element offsets
    pass 2^31 and 2^32 and on both sides of the band's end are those of a short call, and the others zeros."""
    I, dtype = 64, BF16
    band = (1 << 30) // (2 * I // 8)
    R = band + 40
    h, gamma, dact = _make(64, I, dtype, 21)
    spots = [0, (1 << 31) // (2 * I) - 4, (1 << 32) // (2 * I) - 4, band - 4, R - 8]
    want, ck = B.swiglu_forward(h, gamma)
    grads = B.swiglu_backward(dact, ck, gamma)
    q, e = _split(ck, 64, I)
    H = torch.zeros((R, 2 * I), dtype=dtype, device=DEV)
    G = torch.zeros(R, device=DEV)
    D = torch.zeros((R, I), dtype=dtype, device=DEV)
    for n, at in enumerate(spots):
        H[at:at + 8], G[at:at + 8], D[at:at + 8] = h[8 * n:8 * n + 8], gamma[8 * n:8 * n + 8], dact[8 * n:8 * n + 8]
    act, CK = B.swiglu_forward(H, G)
    for n, at in enumerate(spots):
        assert torch.equal(act[at:at + 8], want[8 * n:8 * n + 8]), at
        kept = CK[at * 2 * I:(at + 8) * 2 * I].cpu().numpy().view(np.int8).reshape(8, 2 * I)
        exps = CK[R * 2 * I + at * (I // 16):R * 2 * I + (at + 8) * (I // 16)].cpu().numpy().reshape(8, I // 16)
        assert np.array_equal(kept, q[8 * n:8 * n + 8]) and np.array_equal(exps, e[8 * n:8 * n + 8]), at
    assert int(act.count_nonzero()) == int(want[:40].count_nonzero())
    got = B.swiglu_backward(D, CK, G, act=act)
    for n, at in enumerate(spots):
        for k in ("dh", "act", "dgamma"):
            assert torch.equal(got[k][at:at + 8], grads[k][8 * n:8 * n + 8]), (k, at)
    assert int(got["dh"].count_nonzero()) == int(grads["dh"][:40].count_nonzero())
    # a count below zero, as small as it can be, is no rows in any band
    act.fill_(-776.0)
    B.swiglu_forward(H, G, row_count=torch.tensor([-2 ** 31], dtype=torch.int32, device=DEV), out=act, save=False)
    torch.cuda.synchronize()
    assert bool((act[:64] == -776.0).all()) and bool((act[band - 64:] == -776.0).all())


def test_refusals():
    h, gamma, da = _make(10, 32, BF16, 17)
    _, ck = B.swiglu_forward(h, gamma)
    for bad in (dict(h=h.half()), dict(h=h[:, :33]), dict(h=h.cpu()), dict(gamma=gamma[:9]), dict(gamma=gamma.double()),
                dict(row_count=torch.zeros(2, dtype=torch.int32, device=DEV)), dict(save=False, checkpoint=ck),
                dict(out=da.float()), dict(checkpoint=ck.view(torch.int8))):
        with pytest.raises(ValueError):
            B.swiglu_forward(**(dict(h=h, gamma=gamma) | bad))
    with pytest.raises(B.InklingError) as e:
        B.swiglu_forward(h[:, :48].contiguous())                  # I = 24
    assert e.value.code == B.INKLING_ERR_UNSUPPORTED
    for short in (lambda: B.swiglu_forward(h, checkpoint=ck[:-1]), lambda: B.swiglu_backward(da, ck[:-1])):
        with pytest.raises(B.InklingError) as e:
            short()
        assert e.value.code == B.INKLING_ERR_WORKSPACE
    for bad in (dict(dact=da.float(), dh=h), dict(checkpoint=ck.view(torch.int8)), dict(want_act=False, act=da.clone()),
                dict(dgamma=gamma.double())):
        with pytest.raises(ValueError):
            B.swiglu_backward(**(dict(dact=da, checkpoint=ck) | bad))
    with pytest.raises(B.InklingError) as e:
        B.swiglu_backward(da, ck, act=da)
    assert e.value.code == B.INKLING_ERR_INVALID_ARGUMENT
    assert B.swiglu_forward(h[:0], gamma[:0])[0].shape == (0, 32)
    assert B.swiglu_backward(da[:0], ck, gamma[:0])["dgamma"].shape == (0,)
