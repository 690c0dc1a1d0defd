"""8-bit floating point where its rounding, its ranges and its sums can go wrong: every
e4m3 value and every point between two, more than 2^32 values, the sums of the 8-bit
matrix units by themselves, factors at the ends of fp32's range."""
import sys

import numpy as np
import pytest
import torch

from mixture_experts_feed_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


def _say(msg):
    print(msg, file=sys.stderr, flush=True)


# ---- rounding to e4m3 -----------------------------------------------------------------------


def _every_case(dtype):
    """(value, e4m3 byte): every finite e4m3 number, every point halfway between two of them (to the even one) and
    the numbers of this type next to each of these, of both signs; |value| <= 448."""
    held = [(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10), 8 * e + m) for e in range(16) for m in range(8)][:127]
    assert held[-1] == (448.0, 126) and held[0] == (0.0, 0)
    cases = []
    for (v, byte), (nxt, _) in zip(held, held[1:] + [(None, None)]):
        cases.append((v, byte))
        if nxt is not None:
            mid = (v + nxt) / 2
            cases.append((mid, byte + byte % 2))
            cases += [(_beside(mid, -1, dtype), byte), (_beside(mid, 1, dtype), byte + 1)]
            cases.append((_beside(v, 1, dtype), byte))
            cases.append((_beside(nxt, -1, dtype), byte + 1))
    v, b = np.array([c[0] for c in cases]), np.array([c[1] for c in cases])
    return np.concatenate([v, -v]), np.concatenate([b, b + 128])


def _beside(v, way, dtype):
    """The next fp32 or bf16 number from v >= 0 up or down (from 0 up: the smallest)."""
    if dtype == F32:
        return float(np.nextafter(np.float32(v), np.float32(np.inf if way > 0 else -np.inf)))
    bits = int(np.float32(v).view(np.uint32))
    assert bits % 65536 == 0
    return float(np.uint32(bits + way * 65536).view(np.float32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [0, 40, 118, -60, -126])
def test_every_value_and_every_midpoint(dtype, power):
    """448 in each block makes its scale 2^power, so each other value v is rounded as v / 2^power."""
    v, byte = _every_case(dtype)
    n = -(-v.size // 112 // 16) * 16
    x, want = np.zeros((n, 128)), np.zeros((n, 128), dtype=np.int64)
    x[:, 0], want[:, 0] = 448.0, 126
    for i in range(n):
        some = slice(112 * i, 112 * (i + 1))
        x[i, 1:1 + v[some].size], want[i, 1:1 + v[some].size] = v[some], byte[some]
    x *= 2.0 ** power
    t = torch.from_numpy(x).to(dtype)
    keep = t.double().numpy() == x     # at the smallest scale the type does not hold all of them
    assert keep.all() if power >= 0 else keep[x != 0].mean() > (0.99 if power == -60 else 0.6)
    q, s = B.fp8_quantize_rows(t.to(DEV))
    got = q.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got[keep], want[keep]) and bool((s == 2.0 ** power).all())
    q, s = B.fp8_quantize_weight(t.to(DEV).reshape(n // 16, 16, 128))
    got = q.view(torch.uint8).cpu().numpy().reshape(n, 128)
    assert np.array_equal(got[keep], want[keep]) and bool((s == 2.0 ** power).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_past_32_bits(dtype):
    """Rows and weights of more than 2^32 values: as their parts."""
    R, C, step = 270016, 16384, 16876
    _say(f"quantize {R} x {C} {dtype}")
    assert R * C > 2 ** 32 + 2 ** 20 and R % step == 0
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty((R, C), dtype=dtype, device=DEV)
    for a in range(0, R, step):
        x[a:a + step] = torch.randn((step, C), generator=g, device=DEV)
    v, s = B.fp8_quantize_rows(x)
    for a in range(0, R, step):
        pv, ps = B.fp8_quantize_rows(x[a:a + step])
        assert torch.equal(v[a:a + step].view(torch.uint8), pv.view(torch.uint8)) and torch.equal(s[a:a + step], ps), a
    del v, s
    E, N = 4, R // 4            # 67504 = 527.4 blocks of 128: the last one of each expert is short
    v, s = B.fp8_quantize_weight(x.view(E, N, C))
    for e in range(E):
        pv, ps = B.fp8_quantize_weight(x.view(E, N, C)[e:e + 1])
        assert torch.equal(v[e].view(torch.uint8), pv[0].view(torch.uint8)) and torch.equal(s[e], ps[0]), e
