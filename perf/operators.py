"""The expert-block operators as they are measured: products grouped by expert
with ragged sizes, SwiGLU with its input kept in 8 bits for the backward, and
layer / RMS norm, each in a plain form (elementary torch operations in 32 bits)
and as calls of this package (`own`)."""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # gate_up of one decode step at hidden 6144: 32 tokens, 8 of 128 experts each, weights streamed
        dict(name="expert_up_decode", op="grouped_forward", dtype="bf16", tokens=32, experts=128, top_k=8, n_in=6144,
             n_out=4096, skew=0.0, gather=True),
        # gate_up of a whole prefill batch of the same layer, rows gathered from the token rows
        dict(name="expert_up_prefill", op="grouped_forward", dtype="bf16", tokens=8192, experts=128, top_k=8,
             n_in=6144, n_out=4096, skew=0.1, gather=True),
        # small fp32 experts of odd widths (adapters on experts): the shortest call
        dict(name="expert_adapter_f32", op="grouped_forward", dtype="f32", tokens=333, experts=8, top_k=2, n_in=200,
             n_out=136, skew=0.5, gather=False),
        # both gradients of gate_up in the small bf16 layer, fp32 weight gradients
        dict(name="expert_up_backward", op="grouped_backward", dtype="bf16", tokens=4096, experts=64, top_k=6,
             n_in=2048, n_out=1536, skew=0.3, gather=True, wdtype="f32"),
        # both gradients of the down projections on one GPU of an expert-parallel layer, unevenly loaded
        dict(name="expert_down_backward_shard", op="grouped_backward", dtype="bf16", tokens=1024, experts=16, top_k=8,
             n_in=2048, n_out=6144, skew=1.0, gather=False, wdtype="bf16"),
        # activation between the projections of the prefill batch, forward and backward
        dict(name="swiglu_step_prefill", op="swiglu_step", dtype="bf16", rows=65536, used=65536, inter=2048),
        # the same for a buffer with room left behind the last expert's rows, fp32, odd width
        dict(name="swiglu_step_padded_f32", op="swiglu_step", dtype="f32", rows=1200, used=1003, inter=208),
        # the same for a few rows (adapter tuning on short texts): latency
        dict(name="swiglu_step_short", op="swiglu_step", dtype="bf16", rows=256, used=256, inter=768),
        # the norm before the layer, prefill batch
        dict(name="norm_prefill", op="norm_forward", dtype="bf16", kind="rms", rows=8192, width=6144),
        # ... one decode step
        dict(name="norm_decode", op="norm_forward", dtype="bf16", kind="layer", rows=32, width=6144),
        # its backward over the prefill batch, with the weight's and the bias's gradients
        dict(name="norm_backward_prefill", op="norm_backward", dtype="bf16", kind="layer", rows=8192, width=6144),
        # an odd width in fp32
        dict(name="norm_backward_odd_f32", op="norm_backward", dtype="f32", kind="layer", rows=1001, width=1237),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["grouped_forward", "grouped_backward", "swiglu_step", "norm_forward", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("grouped"):
        c = dict(op=op, dtype=dtype, tokens=_log(rng, 1, 8192), experts=rng.choice([4, 8, 12, 16, 40, 64, 100, 128]),
                 top_k=rng.randint(1, 4), n_in=_log(rng, 64, 6144, 8), n_out=_log(rng, 64, 6144, 8),
                 skew=rng.choice([0.0, 0.2, 0.5]), gather=rng.random() < 0.5)
        if op == "grouped_backward":
            c["wdtype"] = rng.choice(["f32", "bf16"])
        # fp32 matrix rates are a sixteenth of bf16's
        while work(c)["flops"] > (1.6e12 if dtype == "bf16" else 1.0e11):
            c["tokens"] = (c["tokens"] + 1) // 2
        while c["experts"] * c["n_in"] * c["n_out"] > (1 << 30):
            c["n_out"] = max(64, c["n_out"] // 16 * 8)
        return c
    if op == "swiglu_step":
        rows, inter = _log(rng, 1, 65536), _log(rng, 16, 4096, 16)
        rows = max(1, min(rows, 65536 * 2048 // inter // (1 if dtype == "bf16" else 2)))
        used = rows if rng.random() < 0.6 else rng.randint(0, rows)
        return dict(op=op, dtype=dtype, rows=rows, used=max(1, used), inter=inter)
    rows, width = _log(rng, 1, 16384), _log(rng, 8, 12288)
    if rng.random() < 0.6:
        width = max(8, width // 8 * 8)
    rows = max(1, min(rows, 8192 * 6144 // width // (1 if dtype == "bf16" else 2)))
    return dict(op=op, dtype=dtype, kind=rng.choice(["layer", "rms"]), rows=rows, width=width)


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)
    dt, op = TYPES[case["dtype"]], case["op"]
    s = dict(op=op, dt=dt)
    if op.startswith("grouped"):
        T, E, k, K, N = (case[n] for n in ("tokens", "experts", "top_k", "n_in", "n_out"))
        # routing of T tokens: k distinct experts each, some more popular than others; rows sorted by expert
        pop = torch.randn((E,), generator=g, device=DEV) * case["skew"]
        chosen = (torch.randn((T, E), generator=g, device=DEV) + pop).topk(k, dim=1).indices.reshape(-1)
        order = torch.sort(chosen, stable=True).indices
        counts = torch.bincount(chosen, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())   # the plan's largest group
        s["index"] = (order // k).to(torch.int32) if case["gather"] else None
        s["x"] = _randn(g, (T if case["gather"] else T * k, K), dt)
        # one matrix at a time: no fp32 copy of all of them
        s["weight"] = torch.empty((E, N, K), dtype=dt, device=DEV)
        for e in range(E):
            s["weight"][e] = torch.randn((N, K), generator=g, device=DEV) * 0.02
        if op == "grouped_backward":
            s["dout"] = _randn(g, (T * k, N), dt, 0.1)
            s["wdtype"] = TYPES[case["wdtype"]]
    elif op == "swiglu_step":
        R, I = case["rows"], case["inter"]
        # projections of normed tokens: about unit variance, some rows larger
        h = torch.randn((R, 2 * I), generator=g, device=DEV)
        h *= 1.0 + 3.0 * (torch.rand((R, 1), generator=g, device=DEV) < 0.05)
        s["h"] = h.to(dt)
        s["gamma"] = torch.rand((R,), generator=g, device=DEV) * 0.5
        s["dact"] = _randn(g, (R, I), dt, 0.1)
        s["count"] = torch.full((1,), case["used"], dtype=torch.int32, device=DEV)
        # buffers that the call fills as far as rows are used
        s["act"], s["act2"] = torch.zeros((R, I), dtype=dt, device=DEV), torch.zeros((R, I), dtype=dt, device=DEV)
        s["dh"], s["dgamma"] = torch.zeros((R, 2 * I), dtype=dt, device=DEV), torch.zeros((R,), device=DEV)
    else:
        R, H = case["rows"], case["width"]
        s["kind"], s["eps"] = case["kind"], 1e-6
        s["x"] = (torch.randn((R, H), generator=g, device=DEV) * 2.0 + 0.3).to(dt)
        s["weight"] = 1.0 + 0.2 * torch.randn((H,), generator=g, device=DEV)
        s["bias"] = 0.1 * torch.randn((H,), generator=g, device=DEV) if case["kind"] == "layer" else None
        if op == "norm_backward":
            s["dout"] = _randn(g, (R, H), dt, 0.1)
            # what the forward pass kept
            xf = s["x"].double()
            m = xf.mean(1) if case["kind"] == "layer" else torch.zeros((R,), dtype=torch.float64, device=DEV)
            r = 1.0 / torch.sqrt(((xf - m[:, None]) ** 2).mean(1) + s["eps"])
            s["stats"] = torch.stack([m, r], 1).float().contiguous()
    return s


# ---- plain forms ----------------------------------------------------------------------------


def _grid(s):
    """Positions [E, most] of the groups' rows, which of them exist, and each row's place in the grid."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["most"], device=off.device)
    real = at < off[1:, None]
    R = s["dout"].shape[0] if "dout" in s else s["index"].shape[0] if s["index"] is not None else s["x"].shape[0]
    r = torch.arange(R, device=off.device)
    e = torch.searchsorted(off, r, right=True) - 1
    return at.clamp(max=R - 1), real, e * s["most"] + (r - off[e])


def _padded(src, at, real):
    return src[at].float() * real[:, :, None]


def _plain_grouped(s):
    at, real, place = _grid(s)
    rows = at if s["index"] is None else s["index"].long()[at]
    x = _padded(s["x"], rows, real)
    w = s["weight"].float()
    if s["op"] == "grouped_forward":
        y = torch.bmm(x, w.transpose(1, 2))
        return y.reshape(-1, y.shape[2])[place].to(s["dt"])
    d = _padded(s["dout"], at, real)
    dx = torch.bmm(d, w)
    dw = torch.bmm(d.transpose(1, 2), x)
    return {"dx": dx.reshape(-1, dx.shape[2])[place].to(s["dt"]), "dweight": dw.to(s["wdtype"])}


def _plain_swiglu(s):
    R, I = s["dact"].shape
    live = torch.arange(R, device=s["h"].device) < s["count"]
    h = s["h"].float()
    gamma = s["gamma"][:, None]
    act = gamma * (h[:, 0::2] / (1.0 + torch.exp(-h[:, 0::2]))) * h[:, 1::2]
    # 8 bits: one power of two for 32 columns, the smallest that holds the largest value in 127 steps
    b = h.reshape(R, I // 16, 32)
    top = b.abs().amax(2, keepdim=True)
    m, e = torch.frexp(top)                       # top = m 2^e, 0.5 <= m < 1
    e = (e - 7 + (m * 128.0 > 127.0)).clamp(min=-126)
    hq = torch.ldexp(torch.round(torch.ldexp(b, -e)), e).reshape(R, 2 * I)
    g, u = hq[:, 0::2], hq[:, 1::2]
    sg = 1.0 / (1.0 + torch.exp(-g))
    p = g * sg * u
    da = s["dact"].float()
    dp = gamma * da
    dh = torch.stack([dp * u * sg * (1.0 + g * (1.0 - sg)), dp * g * sg], 2).reshape(R, 2 * I)
    keep = live[:, None]
    zero = torch.zeros((), device=h.device)
    return {"act": torch.where(keep, act, zero).to(s["dt"]), "act2": torch.where(keep, gamma * p, zero).to(s["dt"]),
            "dh": torch.where(keep, dh, zero).to(s["dt"]), "dgamma": torch.where(live, (da * p).sum(1), zero)}


def _plain_norm(s):
    x = s["x"].float()
    if s["op"] == "norm_forward":
        m = x.mean(1, keepdim=True) if s["kind"] == "layer" else torch.zeros_like(x[:, :1])
        r = 1.0 / torch.sqrt((x - m).square().mean(1, keepdim=True) + s["eps"])
        y = (x - m) * r * s["weight"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"out": y.to(s["dt"]), "stats": torch.cat([m, r], 1)}
    m, r = s["stats"][:, :1], s["stats"][:, 1:]
    xh = (x - m) * r
    d = s["dout"].float()
    c = d * s["weight"]
    dx = c - xh * (c * xh).mean(1, keepdim=True)
    if s["kind"] == "layer":
        dx = dx - c.mean(1, keepdim=True)
    res = {"dx": (dx * r).to(s["dt"]), "dweight": (d * xh).sum(0)}
    if s["bias"] is not None:
        res["dbias"] = d.sum(0)
    return res


# ---- the package's calls --------------------------------------------------------------------


def _own(s):
    from mixture_experts_feed_amd import binding as B
    op = s["op"]
    if op == "grouped_forward":
        return B.grouped_linear(s["x"], s["weight"], s["offsets"], row_index=s["index"])
    if op == "grouped_backward":
        return {"dx": B.grouped_input_grad(s["dout"], s["weight"], s["offsets"]),
                "dweight": B.grouped_weight_grad(s["dout"], s["x"], s["offsets"], row_index=s["index"],
                                                 weight_grad_dtype=s["wdtype"])}
    if op == "swiglu_step":
        act, kept = B.swiglu_forward(s["h"], s["gamma"], row_count=s["count"], out=s["act"])
        r = B.swiglu_backward(s["dact"], kept, s["gamma"], row_count=s["count"], dh=s["dh"], act=s["act2"],
                              dgamma=s["dgamma"])
        return {"act": act, "act2": r["act"], "dh": r["dh"], "dgamma": r["dgamma"]}
    if op == "norm_forward":
        out, stats = B.norm_forward(s["x"], s["weight"], s["bias"], eps=s["eps"], kind=s["kind"])
        return {"out": out, "stats": stats}
    r = B.norm_backward(s["dout"], s["x"], s["weight"], s["stats"], kind=s["kind"], bias=s["bias"] is not None)
    return {n: r[n] for n in ("dx", "dweight", "dbias") if r[n] is not None}


def run(state):
    if own:
        return _own(state)
    if state["op"].startswith("grouped"):
        return _plain_grouped(state)
    return _plain_swiglu(state) if state["op"] == "swiglu_step" else _plain_norm(state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("grouped"):
        T, E, k, K, N = (case[n] for n in ("tokens", "experts", "top_k", "n_in", "n_out"))
        R = T * k
        met = E * (1.0 - (1.0 - k / E) ** T) if k < E else E   # experts that get a row, evenly chosen
        x = (T if case["gather"] else R) * K * es
        if case["op"] == "grouped_forward":
            return {"bytes": x + met * N * K * es + R * N * es, "flops": 2.0 * R * K * N}
        ws = 2 if case["wdtype"] == "bf16" else 4
        return {"bytes": x + met * N * K * es + R * (N + K) * es + E * N * K * ws, "flops": 4.0 * R * K * N}
    if case["op"] == "swiglu_step":
        U, I = case["used"], case["inter"]
        kept = 2 * I + I / 16      # written once, read once
        return {"bytes": U * (es * 3 * I + kept + kept + es * 4 * I + 12), "flops": U * I * 40.0}
    R, H = case["rows"], case["width"]
    n = 2 if case["op"] == "norm_forward" else 3
    return {"bytes": R * (n * H * es + 8) + 8 * H * (1 if n == 2 else 2), "flops": R * H * (8.0 if n == 2 else 14.0)}


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["op"].startswith("grouped"):
        ends = s["offsets"].tolist()
        src = s["x"] if s["index"] is None else s["x"][s["index"].long()]
        N, K = s["weight"].shape[1:]
        R = src.shape[0]
        if case["op"] == "grouped_forward":
            y = torch.zeros((R, N), dtype=D, device=DEV)
            for e, (a, b) in enumerate(zip(ends, ends[1:])):
                if b > a:
                    torch.mm(src[a:b].to(D), s["weight"][e].to(D).t(), out=y[a:b])
            return y
        dx = torch.zeros((R, K), dtype=D, device=DEV)
        dw = torch.zeros((len(ends) - 1, N, K), dtype=D, device=DEV)
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            if b > a:
                d = s["dout"][a:b].to(D)
                torch.mm(d, s["weight"][e].to(D), out=dx[a:b])
                torch.mm(d.t(), src[a:b].to(D), out=dw[e])
        return {"dx": dx, "dweight": dw}
    if case["op"] == "swiglu_step":
        R, I = s["dact"].shape
        n = case["used"]
        out = {"act": torch.zeros((R, I), dtype=D, device=DEV), "act2": torch.zeros((R, I), dtype=D, device=DEV),
               "dh": torch.zeros((R, 2 * I), dtype=D, device=DEV), "dgamma": torch.zeros((R,), dtype=D, device=DEV)}
        h, gam, da = s["h"][:n].to(D), s["gamma"][:n, None].to(D), s["dact"][:n].to(D)
        out["act"][:n] = gam * h[:, 0::2] * torch.sigmoid(h[:, 0::2]) * h[:, 1::2]
        blocks = h.unflatten(1, (-1, 32))
        need = blocks.abs().amax(-1, keepdim=True) / 127.0
        step = torch.exp2(torch.ceil(torch.log2(need.clamp(min=2.0 ** -126))))
        step = torch.where(step / 2 >= need.clamp(min=2.0 ** -126), step / 2, step)   # a logarithm rounded up
        step = torch.where(step < need, step * 2, step)                               # ... or down
        back = ((blocks / step).round() * step).flatten(1)
        gate, up = back[:, 0::2], back[:, 1::2]
        sig = torch.sigmoid(gate)
        out["act2"][:n] = gam * gate * sig * up
        out["dgamma"][:n] = (da * gate * sig * up).sum(1)
        out["dh"][:n, 0::2] = gam * da * up * (sig + gate * sig * (1.0 - sig))
        out["dh"][:n, 1::2] = gam * da * gate * sig
        return out
    x, w = s["x"].to(D), s["weight"].to(D)
    H = x.shape[1]
    if case["op"] == "norm_forward":
        mean = x.sum(1) / H if case["kind"] == "layer" else torch.zeros_like(x[:, 0])
        inv = torch.rsqrt((x - mean[:, None]).pow(2).sum(1) / H + s["eps"])
        y = w * (x - mean[:, None]) * inv[:, None] + (0.0 if s["bias"] is None else s["bias"].to(D))
        return {"out": y, "stats": torch.stack([mean, inv], 1)}
    mean, inv = s["stats"][:, 0].to(D), s["stats"][:, 1].to(D)
    d = s["dout"].to(D)
    unit = (x - mean[:, None]) * inv[:, None]
    proj = (d * w * unit).sum(1, keepdim=True) / H
    if case["kind"] == "layer":
        dx = inv[:, None] * (d * w - (d @ w)[:, None] / H - unit * proj)
    else:
        dx = inv[:, None] * (d * w - unit * proj)
    res = {"dx": dx, "dweight": torch.einsum("rh,rh->h", d, unit)}
    if s["bias"] is not None:
        res["dbias"] = d.sum(0)
    return res
