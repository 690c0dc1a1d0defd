"""The expert-block operators together, as a training step and a decode step use
them: norm -> inkling_moe_route -> grouped gate_up (rows gathered through the
routing) -> SwiGLU with the 8-bit checkpoint -> grouped down -> sum over the
chosen experts, and back.

Forward and gradients are compared with 64-bit numpy that takes the routing and
the checkpoint's own bytes as they are (both are tested on their own), so that
what is left is bf16 rounding: every stage rounds its result once, a relative
error of at most 2^-8 a value.  A value that passed s stages on its way and was
summed from terms t is off by at most s 2^-8 sum|t| to first order, where the
sum runs over the whole chain of absolute values; the bars below count the
stages and take that sum from the reference's absolute chain.  (fp32 sums add
less than 2^-13 of it.)
"""
import sys

import numpy as np
import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _f64(t):
    return t.detach().cpu().double().numpy()


def _sig(g):
    return 1.0 / (1.0 + np.exp(-g))


def _layer(T, H, E, k, I, seed=1, pad=None):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, sc=1.0: (torch.randn(s, generator=g) * sc)  # noqa: E731
    p = dict(x=rn(T, H).to(BF16).to(DEV), nw=(1 + 0.1 * rn(H)).to(DEV), bank=rn(E, H, sc=0.05).to(DEV),
             bias=rn(E, sc=0.01).to(DEV), wgu=rn(E, 2 * I, H, sc=0.05).to(BF16).to(DEV),
             wd=rn(E, H, I, sc=0.05).to(BF16).to(DEV), dout=rn(T, H).to(BF16).to(DEV), k=k)
    p["pad"] = pad
    return p


def _forward(p, keep=True):
    T, H = p["x"].shape
    k = p["k"]
    n, stats = B.norm_forward(p["x"], p["nw"], kind="rms", eps=1e-6)
    r = B.route(n, p["bank"], p["bias"], k, 2.0, 1.0, padding_mask=p["pad"])
    off, slots = r["expert_offsets"], r["sorted_slots"]
    token = torch.div(slots, k, rounding_mode="floor").to(torch.int32)
    gamma = r["topk_weights"].reshape(-1)[slots.long().clamp(min=0)].contiguous()
    E = off.shape[0] - 1
    count = off[E:]
    h = B.grouped_linear(n, p["wgu"], off, row_index=token)
    act, ck = B.swiglu_forward(h, gamma, row_count=count, save=keep)
    y = B.grouped_linear(act, p["wd"], off, out=torch.zeros((T * k, H), dtype=BF16, device=DEV))
    live = torch.arange(T * k, device=DEV) < count
    out = torch.zeros((T, H), device=DEV).index_add_(0, token.long().clamp(min=0), y.float() * live[:, None])
    return dict(n=n, stats=stats, off=off, token=token, gamma=gamma, h=h, act=act, ck=ck, y=y, out=out, count=count,
                live=live, routing=r)


def _backward(p, f):
    T, H = p["x"].shape
    dy = p["dout"][f["token"].long().clamp(min=0)].contiguous()
    da = B.grouped_input_grad(dy, p["wd"], f["off"])
    s = B.swiglu_backward(da, f["ck"], f["gamma"], row_count=f["count"])
    dwd = B.grouped_weight_grad(dy, s["act"], f["off"])
    dwgu = B.grouped_weight_grad(s["dh"], f["n"], f["off"], row_index=f["token"])
    dxr = B.grouped_input_grad(s["dh"], p["wgu"], f["off"])
    dn = torch.zeros((T, H), device=DEV).index_add_(0, f["token"].long().clamp(min=0),
                                                    torch.where(f["live"][:, None], dxr.float(), 0.0)).to(BF16)
    g = B.norm_backward(dn, p["x"], p["nw"], f["stats"], kind="rms")
    return dict(dwd=dwd, dwgu=dwgu, dgamma=s["dgamma"], dn=dn, dx=g["dx"], dnw=g["dweight"])


def _within(name, got, want, chain, stages):
    err = np.abs(_f64(got) - want)
    bound = stages * 2.0 ** -8 * chain * 1.05 + 1e-30
    assert (err <= bound).all(), f"{name}: worst {np.max(err / bound):.2f} of the bound"


@pytest.mark.parametrize("shape", [(200, 256, 16, 4, 128), (37, 192, 5, 2, 48), (700, 320, 3, 1, 208),
                                   (24, 512, 64, 6, 96)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("padded", [False, True], ids=["", "padded"])
def test_training_step(shape, padded):
    T, H, E, k, I = shape
    pad = None
    if padded:
        pad = torch.zeros(T, dtype=torch.uint8, device=DEV)
        pad[T // 3::4] = 1
    p = _layer(*shape, seed=T, pad=pad)
    f = _forward(p)
    b = _backward(p, f)
    torch.cuda.synchronize()
    n, off, tok = _f64(f["n"]), f["off"].cpu().numpy(), f["token"].cpu().numpy()
    R = int(off[-1])
    assert R == T * k if not padded else R < T * k
    gam, wgu, wd = _f64(f["gamma"])[:, None], _f64(p["wgu"]), _f64(p["wd"])
    # the values that the checkpoint gives back
    raw = f["ck"].cpu().numpy()
    q = raw[:T * k * 2 * I].view(np.int8).reshape(T * k, 2 * I).astype(np.float64)
    e = raw[T * k * 2 * I:T * k * 2 * I + T * k * (I // 16)].reshape(T * k, I // 16).astype(np.float64) - 127
    hq = q * np.repeat(np.exp2(e), 32, axis=1)
    # forward from the normed rows
    out, chain = np.zeros((T, H)), np.zeros((T, H))
    h64 = np.zeros((T * k, 2 * I))
    for i in range(E):
        rows = slice(off[i], off[i + 1])
        h = n[tok[rows]] @ wgu[i].T
        h64[rows] = h
        ha = np.abs(n[tok[rows]]) @ np.abs(wgu[i]).T
        g, u = h[:, 0::2], h[:, 1::2]
        act = gam[rows] * g * _sig(g) * u
        # |d act| for relative errors of g and u of their own chains
        aa = np.abs(gam[rows]) * (np.abs(u) * ha[:, 0::2] * 1.1 + ha[:, 1::2] * np.abs(g) * _sig(g)) + np.abs(act)
        np.add.at(out, tok[rows], act @ wd[i].T)
        np.add.at(chain, tok[rows], aa @ np.abs(wd[i]).T)
    _within("out", f["out"], out, chain, 3)
    assert (np.abs(hq[:R] - _f64(f["h"])[:R]).reshape(R, -1, 32).max(2)
            <= np.abs(_f64(f["h"])[:R]).reshape(R, -1, 32).max(2) / 127).all()
    # backward from the checkpoint's values
    d = _f64(p["dout"])
    dn, dnc = np.zeros((T, H)), np.zeros((T, H))
    for i in range(E):
        rows = slice(off[i], off[i + 1])
        if off[i] == off[i + 1]:
            assert int(b["dwd"][i].count_nonzero()) == 0 and int(b["dwgu"][i].count_nonzero()) == 0
            continue
        dy = d[tok[rows]]
        da, daa = dy @ wd[i], np.abs(dy) @ np.abs(wd[i])
        g, u = hq[rows, 0::2], hq[rows, 1::2]
        s = _sig(g)
        pp = g * s * u
        slope = u * s * (1 + g * (1 - s))
        dh, dhc = np.empty((len(dy), 2 * I)), np.empty((len(dy), 2 * I))
        dh[:, 0::2], dh[:, 1::2] = gam[rows] * da * slope, gam[rows] * da * g * s
        dhc[:, 0::2], dhc[:, 1::2] = np.abs(gam[rows]) * daa * np.abs(slope), np.abs(gam[rows]) * daa * np.abs(g) * s
        _within("dgamma", b["dgamma"][rows], (da * pp).sum(1), (daa * np.abs(pp)).sum(1), 2)
        _within("dwd", b["dwd"][i], dy.T @ (gam[rows] * pp), np.abs(dy).T @ np.abs(gam[rows] * pp), 2)
        _within("dwgu", b["dwgu"][i], dh.T @ n[tok[rows]], dhc.T @ np.abs(n[tok[rows]]), 3)
        np.add.at(dn, tok[rows], dh @ wgu[i])
        np.add.at(dnc, tok[rows], dhc @ np.abs(wgu[i]))
    _within("dn", b["dn"], dn, dnc, 4)
    # the norm's backward at the gradient it was given
    x, nw, dn1, r = _f64(p["x"]), _f64(p["nw"]), _f64(b["dn"]), _f64(f["stats"])[:, 1:]
    xh = x * r
    c = dn1 * nw
    dx = r * (c - xh * (c * xh).mean(1, keepdims=True))
    _within("dx", b["dx"], dx, np.abs(dx) + r * 2.0 ** -8 * (np.abs(c) + np.abs(xh) * np.abs(c * xh).mean(1, keepdims=True)), 1)
    _within("dnw", b["dnw"], (dn1 * xh).sum(0), np.abs(dn1 * xh).sum(0), 1)


def test_against_the_layer():
    """The pieces give what the fused layer gives for the same weights (no shared
    experts): both are within bf16 rounding of the same sums."""
    p = _layer(300, 256, 16, 4, 128, seed=3)
    f = _forward(p, keep=False)
    out, r = B.forward(f["n"], p["bank"], p["bias"], p["wgu"], p["wd"], None, None, 4, 2.0, 1.0, return_routing=True,
                       out_dtype=F32)
    torch.cuda.synchronize()
    assert torch.equal(r["sorted_slots"], f["routing"]["sorted_slots"])
    rms = float(out.square().mean().sqrt())
    # h, act and y rounded to bf16 here; four of 4 experts' rows summed
    assert float((out - f["out"]).abs().max()) <= 8 * 2.0 ** -8 * rms * 4


def test_decode_step_in_a_graph():
    """One to 32 tokens, captured once for the largest batch; a smaller batch is
    the same graph with its other tokens masked out."""
    p = _layer(32, 256, 32, 4, 128, seed=5, pad=torch.zeros(32, dtype=torch.uint8, device=DEV))
    T, H, k = 32, 256, 4
    E, I = 32, 128
    dims = B.make_dims(T, H, E, k, 0, 64, BF16)
    ws = B.alloc_workspace(dims, DEV)
    bufs = dict(n=torch.empty((T, H), dtype=BF16, device=DEV), h=torch.zeros((T * k, 2 * I), dtype=BF16, device=DEV),
                act=torch.zeros((T * k, I), dtype=BF16, device=DEV), y=torch.zeros((T * k, H), dtype=BF16, device=DEV))
    res = {}

    def step():
        B.norm_forward(p["x"], p["nw"], kind="rms", out=bufs["n"], save=False)
        r = B.route(bufs["n"], p["bank"], p["bias"], k, 2.0, 1.0, padding_mask=p["pad"], workspace=ws)
        token = torch.div(r["sorted_slots"], k, rounding_mode="floor").to(torch.int32)
        gamma = r["topk_weights"].reshape(-1)[r["sorted_slots"].long().clamp(min=0)].contiguous()
        off = r["expert_offsets"]
        B.grouped_linear(bufs["n"], p["wgu"], off, row_index=token, out=bufs["h"])
        B.swiglu_forward(bufs["h"], gamma, row_count=off[E:], out=bufs["act"], save=False)
        B.grouped_linear(bufs["act"], p["wd"], off, out=bufs["y"])
        res["off"], res["token"] = off, token

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for tokens in (32, 1, 7, 32):
        p["pad"].fill_(1)
        p["pad"][:tokens] = 0
        p["x"].copy_(torch.randn((T, H), generator=torch.Generator().manual_seed(tokens)).to(BF16))
        g.replay()
        torch.cuda.synchronize()
        off, tok = res["off"].cpu().numpy(), res["token"].cpu().numpy()
        assert off[-1] == tokens * k
        got = bufs["y"][:tokens * k].clone()
        f = _forward(p, keep=False)
        torch.cuda.synchronize()
        assert torch.equal(f["y"][:tokens * k], got)
