"""Operators around the experts as they are measured: tokens sorted by expert and
back with the routing weights applied, its gradients, and products grouped by
expert in 8-bit floating point with a scale for each block of 128, each in a
plain form (elementary torch operations in 32 bits) and as calls of this package
(`own`)."""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
BLOCK = 128


def listed():
    return [
        # one decode step: 32 tokens of hidden 6144 to their 8 of 128 experts, as rows sorted by expert
        dict(name="dispatch_decode", op="dispatch", dtype="bf16", tokens=32, experts=128, top_k=8, width=6144, skew=0.0,
             pad=0.0, weighted=False),
        # a prefill batch of the same layer, an eighth of its tokens padding
        dict(name="dispatch_prefill", op="dispatch", dtype="bf16", tokens=8192, experts=128, top_k=8, width=6144,
             skew=0.2, pad=0.125, weighted=False),
        # small fp32 layer of an odd width that applies the routing weights to the expert's input
        dict(name="dispatch_odd_f32", op="dispatch", dtype="f32", tokens=1001, experts=12, top_k=2, width=1237,
             skew=0.5, pad=0.0, weighted=True),
        # the experts' rows of a decode step back to the tokens, on top of the shared experts' output
        dict(name="combine_decode", op="combine", dtype="bf16", tokens=32, experts=128, top_k=8, width=6144, skew=0.0,
             pad=0.0),
        # ... of the prefill batch
        dict(name="combine_prefill", op="combine", dtype="bf16", tokens=8192, experts=128, top_k=8, width=6144,
             skew=0.2, pad=0.125),
        # a training step of the prefill batch: gradients of the combine and of the dispatch
        dict(name="sorting_backward_prefill", op="sorting_backward", dtype="bf16", tokens=8192, experts=128, top_k=8,
             width=6144, skew=0.2, pad=0.0),
        # the same for a small fp32 layer of an odd width
        dict(name="sorting_backward_odd_f32", op="sorting_backward", dtype="f32", tokens=1001, experts=12, top_k=2,
             width=1237, skew=0.5, pad=0.1),
        # gate_up of one decode step with 8-bit weights, which are streamed
        dict(name="fp8_up_decode", op="fp8_forward", dtype="bf16", tokens=32, experts=128, top_k=8, n_in=6144,
             n_out=4096, skew=0.0),
        # gate_up of the prefill batch, rows gathered from the token rows
        dict(name="fp8_up_prefill", op="fp8_forward", dtype="bf16", tokens=8192, experts=128, top_k=8, n_in=6144,
             n_out=4096, skew=0.1),
        # one dense projection of a single token (the shared expert of a chat with one user)
        dict(name="fp8_single_token", op="fp8_forward", dtype="bf16", tokens=1, experts=1, top_k=1, n_in=6144,
             n_out=4096, skew=0.0),
        # the input gradient of gate_up in the small layer, 8-bit output gradients
        dict(name="fp8_up_backward", op="fp8_backward", dtype="bf16", tokens=4096, experts=64, top_k=6, n_in=2048,
             n_out=1536, skew=0.3),
        # the same on one GPU of an expert-parallel layer, unevenly loaded
        dict(name="fp8_down_backward_shard", op="fp8_backward", dtype="bf16", tokens=1024, experts=16, top_k=8,
             n_in=2048, n_out=6144, skew=1.0),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "sorting_backward", "fp8_forward", "fp8_forward", "fp8_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    experts = rng.choice([1, 4, 8, 12, 16, 40, 64, 100, 128])
    c = dict(op=op, dtype=dtype, tokens=_log(rng, 1, 8192), experts=experts, top_k=min(experts, rng.randint(1, 8)),
             skew=rng.choice([0.0, 0.2, 0.5]))
    if op.startswith("fp8"):
        c["n_in"], c["n_out"] = _log(rng, 64, 6144, 16), _log(rng, 64, 6144, 16)
        while work(c)["flops"] > 3.2e12:
            c["tokens"] = (c["tokens"] + 1) // 2
        while c["experts"] * c["n_in"] * c["n_out"] > (1 << 30):
            c["n_out"] = max(64, c["n_out"] // 32 * 16)
        return c
    width = _log(rng, 8, 6144)
    c["width"] = width if rng.random() < 0.4 else max(8, width // 8 * 8)
    c["pad"] = rng.choice([0.0, 0.0, 0.1, 0.3])
    if op == "dispatch":
        c["weighted"] = rng.random() < 0.4
    if dtype == "f32":
        c["tokens"] = (c["tokens"] + 1) // 2
    return c


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _routing(s, case, g):
    """k distinct experts a token, some more popular than others; padded tokens; the rows' order."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    pop = torch.randn((E,), generator=g, device=DEV) * case["skew"]
    topk = (torch.randn((T, E), generator=g, device=DEV) + pop).topk(k, dim=1).indices.to(torch.int32).contiguous()
    mask = None
    if case.get("pad", 0.0) > 0.0:
        mask = (torch.rand((T,), generator=g, device=DEV) < case["pad"]).to(torch.uint8)
    s.update(E=E, topk=topk, mask=mask)
    if case["op"] == "dispatch":
        return
    key = topk.reshape(-1).long()
    if mask is not None:
        key = torch.where(mask.repeat_interleave(k) != 0, E, key)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    used = int(counts.sum())
    pos = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    pos[order[:used]] = torch.arange(used, dtype=torch.int32, device=DEV)
    s.update(positions=pos.reshape(T, k), used=used, most=int(counts.max()), index=(order // k).to(torch.int32))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 29)
    dt, op = TYPES[case["dtype"]], case["op"]
    T, k = case["tokens"], case["top_k"]
    s = dict(op=op, dt=dt)
    _routing(s, case, g)
    if not op.startswith("fp8"):
        H = case["width"]
        # routing weights of k experts, as of a softmax
        w = torch.softmax(torch.randn((T, k), generator=g, device=DEV), 1).contiguous()
        if op == "dispatch":
            s["x"] = _randn(g, (T, H), dt)
            s["weights"] = w if case["weighted"] else None
            # the buffer that the call fills as far as rows are used
            s["rows"] = torch.zeros((T * k, H), dtype=dt, device=DEV)
        elif op == "combine":
            s.update(rows=_randn(g, (T * k, H), dt, 0.3), weights=w, addend=_randn(g, (T, H), dt))
        else:
            s.update(rows=_randn(g, (T * k, H), dt, 0.3), weights=w, dout=_randn(g, (T, H), dt, 0.1),
                     dgathered=_randn(g, (T * k, H), dt, 0.1), drows=torch.zeros((T * k, H), dtype=dt, device=DEV))
        return s
    E, K, N = case["experts"], case["n_in"], case["n_out"]
    # 8-bit weights with a scale for each block of 128 x 128, as a checkpoint holds them
    s["weight"] = torch.empty((E, N, K), dtype=E4M3, device=DEV)
    for e in range(E):
        s["weight"][e] = (torch.randn((N, K), generator=g, device=DEV) * 110.0).clamp(-448.0, 448.0).to(E4M3)
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    s["wscale"] = (0.5 + torch.rand((E, nb, kb), generator=g, device=DEV)) * (0.02 / 110.0)
    if op == "fp8_forward":
        # token rows, some larger than others, a few columns far larger (as hidden states have them)
        x = torch.randn((T, K), generator=g, device=DEV) * (1.0 + 3.0 * (torch.rand((T, 1), generator=g, device=DEV) < 0.05))
        x *= 1.0 + 20.0 * (torch.rand((1, K), generator=g, device=DEV) < 0.002)
        s["x"] = x.to(dt)
    else:
        s["dout"] = _randn(g, (T * k, N), dt, 0.1)
    return s


# ---- plain forms ----------------------------------------------------------------------------


def _plain_order(topk, mask, E):
    T, k = topk.shape
    key = topk.reshape(-1).long()
    if mask is not None:
        key = torch.where(mask.repeat_interleave(k) != 0, E, key)
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(E, device=key.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    r = torch.arange(T * k, device=key.device)
    slots = torch.where(r < offsets[E], order, -1)
    pos = torch.empty_like(r)
    pos[order] = torch.where(r < offsets[E], r, -1)
    return {"offsets": offsets.to(torch.int32), "slots": slots.to(torch.int32),
            "positions": pos.reshape(T, k).to(torch.int32)}


def _plain_dispatch(s):
    o = _plain_order(s["topk"], s["mask"], s["E"])
    k = s["topk"].shape[1]
    live = (o["slots"] >= 0)[:, None]
    slot = o["slots"].long().clamp(min=0)
    rows = s["x"].float()[slot // k]
    if s["weights"] is not None:
        rows = rows * s["weights"].reshape(-1)[slot][:, None]
    o["rows"] = torch.where(live, rows, torch.zeros((), device=rows.device)).to(s["dt"])
    return o


def _taken(rows, positions):
    """[T, k, H] rows of each token in 32 bits, zero where a slot has none."""
    live = (positions >= 0)[:, :, None]
    return torch.where(live, rows[positions.long().clamp(min=0)].float(), torch.zeros((), device=rows.device))


def _plain_combine(s):
    return (s["addend"].float() + (s["weights"][:, :, None] * _taken(s["rows"], s["positions"])).sum(1)).to(s["dt"])


def _plain_sorting_backward(s):
    pos, d = s["positions"], s["dout"].float()
    T, k = pos.shape
    got = _taken(s["rows"], pos)
    dweights = (got * d[:, None, :]).sum(2)
    dx = _taken(s["dgathered"], pos).sum(1).to(s["dt"])
    # each row's slot; rows that no slot has stay zero
    slot = torch.full((T * k + 1,), -1, dtype=torch.long, device=pos.device)
    flat = pos.reshape(-1).long()
    slot[torch.where(flat >= 0, flat, T * k)] = torch.arange(T * k, device=pos.device)
    slot = slot[:-1]
    at = slot.clamp(min=0)
    drows = torch.where((slot >= 0)[:, None], s["weights"].reshape(-1)[at][:, None] * d[at // k],
                        torch.zeros((), device=pos.device))
    return {"drows": drows.to(s["dt"]), "dweights": dweights, "dx": dx}


def _blocks(x):
    """x [.., n] in blocks of 128 columns, the last one filled up with zeros."""
    n = x.shape[-1]
    return torch.nn.functional.pad(x, (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))


def _through_8_bits(x):
    """x [R, n] as e4m3 with one power of two for 128 columns gives it back: the smallest that holds the
    block's largest value in 448 steps."""
    b = _blocks(x.float())
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))      # largest = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875)).clamp(min=-126)
    q = torch.ldexp(b, -e).to(E4M3).float()
    return torch.ldexp(q, e).flatten(-2)[..., :x.shape[-1]]


def _weight32(s):
    w = s["weight"]
    E, N, K = w.shape
    scale = s["wscale"].repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    return w.float() * scale


def _plain_fp8(s):
    off = s["offsets"].long()
    R = s["index"].shape[0]
    at = (off[:-1, None] + torch.arange(s["most"], device=off.device))
    real = at < off[1:, None]
    at = at.clamp(max=R - 1)
    r = torch.arange(R, device=off.device)
    e = torch.searchsorted(off, r, right=True) - 1
    place = e * s["most"] + (r - off[e])
    w = _weight32(s)
    if s["op"] == "fp8_forward":
        x = _through_8_bits(s["x"])[s["index"].long()[at]] * real[:, :, None]
        y = torch.bmm(x, w.transpose(1, 2).contiguous())
    else:
        y = torch.bmm(_through_8_bits(s["dout"])[at] * real[:, :, None], w)
    return y.flatten(0, 1)[place].to(s["dt"])


# ---- the package's calls --------------------------------------------------------------------


def _own(s):
    from mixture_experts_feed_amd import binding as B
    op = s["op"]
    if op == "dispatch":
        o = B.expert_order(s["topk"], s["E"], padding_mask=s["mask"])
        rows = B.dispatch_forward(s["x"], o["positions"], weights=s["weights"], rows=s["rows"])
        return {"offsets": o["expert_offsets"], "slots": o["sorted_slots"], "positions": o["positions"], "rows": rows}
    if op == "combine":
        return B.combine_forward(s["rows"], s["positions"], weights=s["weights"], addend=s["addend"])
    if op == "sorting_backward":
        g = B.combine_backward(s["dout"], s["positions"], rows=s["rows"], weights=s["weights"], drows=s["drows"])
        d = B.dispatch_backward(s["dgathered"], s["positions"])
        return {"drows": g["drows"], "dweights": g["dweights"], "dx": d["dx"]}
    if op == "fp8_forward":
        x8, xs = B.fp8_quantize_rows(s["x"])
        return B.fp8_grouped_linear(x8, xs, s["weight"], s["wscale"], s["offsets"], row_index=s["index"],
                                    out_dtype=s["dt"])
    d8, ds = B.fp8_quantize_rows(s["dout"])
    return B.fp8_grouped_input_grad(d8, ds, s["weight"], s["wscale"], s["offsets"], dx_dtype=s["dt"])


def run(state):
    if own:
        return _own(state)
    if state["op"].startswith("fp8"):
        return _plain_fp8(state)
    return {"dispatch": _plain_dispatch, "combine": _plain_combine,
            "sorting_backward": _plain_sorting_backward}[state["op"]](state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    R = T * k
    if case["op"].startswith("fp8"):
        K, N = case["n_in"], case["n_out"]
        met = E * (1.0 - (1.0 - k / E) ** T) if k < E else E   # experts that get a row, evenly chosen
        rows = T * K * es + R * N * es if case["op"] == "fp8_forward" else R * (N + K) * es
        return {"bytes": rows + met * N * K * (1.0 + 4.0 / BLOCK ** 2) + 8.0 * R, "flops": 2.0 * R * K * N}
    H, U = case["width"], R * (1.0 - case["pad"])
    if case["op"] == "dispatch":
        return {"bytes": (T * H + U * H) * es + 12.0 * R + 4 * E + (4.0 * R if case["weighted"] else 0.0),
                "flops": 1.0 * U * H}
    if case["op"] == "combine":
        return {"bytes": (2 * T * H + U * H) * es + 8.0 * R, "flops": 2.0 * U * H}
    return {"bytes": (2 * T * H + 3 * U * H) * es + 12.0 * R, "flops": 4.0 * U * H}


# ---- the definition in 64 bits --------------------------------------------------------------


def _exact_8_bits(x):
    """e4m3 by its definition: 3 fraction bits, exponents from -6, on values scaled to at most 448."""
    R, n = x.shape
    out = torch.empty((R, n), dtype=torch.float64, device=x.device)
    for c in range(0, n, BLOCK):
        b = x[:, c:c + BLOCK].double()
        need = (b.abs().amax(1, keepdim=True) / 448.0).clamp(min=2.0 ** -126)
        scale = torch.exp2(torch.ceil(torch.log2(need)))
        scale = torch.where(scale / 2 >= need, scale / 2, scale)    # a logarithm rounded up
        scale = torch.where(scale < need, scale * 2, scale)         # ... or down
        v = b / scale
        top = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))))
        top = torch.where(top * 2 <= v.abs(), top * 2, torch.where((top > v.abs()) & (top > 2.0 ** -6), top / 2, top))
        step = top / 8.0
        out[:, c:c + BLOCK] = (v / step).round() * step * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    op, T, k = case["op"], case["tokens"], case["top_k"]
    if op.startswith("fp8"):
        ends = s["offsets"].tolist()
        E, N, K = s["weight"].shape
        src = _exact_8_bits(s["x"])[s["index"].long()] if op == "fp8_forward" else _exact_8_bits(s["dout"])
        y = torch.zeros((src.shape[0], N if op == "fp8_forward" else K), dtype=D, device=DEV)
        n_at, k_at = torch.arange(N, device=DEV) // BLOCK, torch.arange(K, device=DEV) // BLOCK
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            if b > a:
                w = s["weight"][e].to(D) * s["wscale"][e].to(D)[n_at][:, k_at]
                torch.mm(src[a:b], w.t() if op == "fp8_forward" else w, out=y[a:b])
        return y
    if op == "dispatch":
        # slots in order of (expert, slot), from the host
        topk, mask = s["topk"].tolist(), None if s["mask"] is None else s["mask"].tolist()
        lists = [[] for _ in range(s["E"])]
        for t, chosen in enumerate(topk):
            if mask is None or not mask[t]:
                for i, e in enumerate(chosen):
                    lists[e].append(t * k + i)
        offsets, slots = [0], []
        for one in lists:
            slots += one
            offsets.append(len(slots))
        pos = [-1] * (T * k)
        for r, sl in enumerate(slots):
            pos[sl] = r
        rows = torch.zeros((T * k, case["width"]), dtype=D, device=DEV)
        at = torch.tensor(slots, dtype=torch.long, device=DEV)
        rows[:len(slots)] = s["x"].to(D)[torch.div(at, k, rounding_mode="floor")]
        if s["weights"] is not None:
            rows[:len(slots)] *= s["weights"].to(D).flatten()[at].unsqueeze(1)
        slots += [-1] * (T * k - len(slots))
        return {"offsets": torch.tensor(offsets, dtype=torch.int32, device=DEV),
                "slots": torch.tensor(slots, dtype=torch.int32, device=DEV),
                "positions": torch.tensor(pos, dtype=torch.int32, device=DEV).reshape(T, k), "rows": rows}
    pos, w = s["positions"].long(), s["weights"].to(D)
    if op == "combine":
        out = s["addend"].to(D)
        for i in range(k):
            t = torch.nonzero(pos[:, i] >= 0).flatten()
            out[t] += w[t, i, None] * s["rows"][pos[t, i]].to(D)
        return out
    d = s["dout"].to(D)
    dx, drows = torch.zeros_like(d), torch.zeros(s["rows"].shape, dtype=D, device=DEV)
    dw = torch.zeros((T, k), dtype=D, device=DEV)
    for i in range(k):
        t = torch.nonzero(pos[:, i] >= 0).flatten()
        p = pos[t, i]
        dx[t] += s["dgathered"][p].to(D)
        drows[p] = w[t, i, None] * d[t]
        dw[t, i] = torch.linalg.vecdot(s["rows"][p].to(D), d[t])
    return {"drows": drows, "dweights": dw, "dx": dx}
