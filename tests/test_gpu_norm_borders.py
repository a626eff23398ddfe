"""The norm's rows next to the border between two values of their type: one rounding from
the 64-bit y to bf16, and one to e4m3.

Every y is m (1 + d), m half way between two neighbours, with |d| far below a step of fp32:
t w = 3 m from two factors of few bits, and eps makes the row's factor (1 + d) / 3. What the
kernel holds in 64 bits is off by less than 2^-48, d is 2^-27 to 2^-40. It is the neighbour
on d's side that is nearest."""
import pytest
import torch

import combine_moe_route_03_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
OFFS = [s * 2.0 ** -p for p in (27, 33, 40) for s in (1, -1)]


def factors(odd):
    """(m, a, b) with 3 m = a b, a and b of up to 8 bits, for those odd numbers that have some."""
    out = []
    for m in odd:
        a = next((a for a in range(1, 256) if 3 * m % a == 0 and 3 * m // a < 256), None)
        if a is not None:
            out.append((m, a, 3 * m // a))
    return out


def row(cases, H, dtype):
    """t, w and m of H columns from (m, t, w); both signs, the cases over and over."""
    t, w, m = (torch.tensor(v, dtype=torch.float64) for v in zip(*[(a, b, y) for y, a, b in cases]))
    n = torch.arange(H) % (2 * len(cases))
    sign = torch.where(n < len(cases), 1.0, -1.0).double()
    n = n % len(cases)
    t, w, m = t[n] * sign, w[n], m[n] * sign
    assert torch.equal(t, t.to(dtype).double()) and torch.equal(w, w.to(dtype).double())
    assert torch.equal(t * w, 3 * m)
    return t, w, m


def norm(t, w, off, T, dtype, **kw):
    eps = 9.0 / (1 + off) ** 2 - float((t * t).mean())
    assert eps > 0
    return moe.add_rms_norm(t.to(dtype).to(DEV).repeat(T, 1), w.to(dtype).to(DEV), eps, **kw)


@pytest.mark.parametrize("T,H", [(1, 128), (3, 512), (2, 4096), (1030, 144), (1027, 1024), (2, 20480)])
@pytest.mark.parametrize("where", ["normal", "subnormal", "largest"])
def test_bf16(where, T, H):
    """9-bit odd numbers, half way between two of 8 bits; odd multiples of half the smallest
    step; half way between the largest number and infinity."""
    if where == "normal":
        cases = [(float(m), a * 2.0 ** -8, b * 2.0 ** 8) for m, a, b in factors(range(257, 512, 2))]
        unit = 1.0
    elif where == "subnormal":
        cases = [(m * 2.0 ** -134, a * 2.0 ** -8, b * 2.0 ** -126) for m, a, b in factors(range(1, 254, 2))]
        unit = 2.0 ** -134
    else:
        # seven zeros for each: the mean of the squares stays below 9
        cases, unit = [(511 * 2.0 ** 119, 21 / 4, 73 * 2.0 ** 121)] + [(0.0, 0.0, 0.0)] * 7, 2.0 ** 119
    t, w, m = row(cases, H, BF16)
    for off in OFFS:
        got = norm(t, w, off, T, BF16)[1].double().cpu()
        want = m + m.sign() * (unit if off > 0 else -unit)
        want[want.abs() >= 2.0 ** 128] *= float("inf")
        bad = (got != want).any(0).nonzero().flatten().tolist()
        assert not bad, f"{off}: {len(bad)} of {H} columns: {[(float(m[i]), float(got[0, i])) for i in bad[:4]]}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,shift,size", [(1, 128, 0, 0.75), (3, 512, 0, 0.75), (1030, 256, 0, 0.75),
                                            (1027, 1024, 0, 0.75), (2, 20480, 0, 0.75), (2, 256, -126, 0.375),
                                            (1, 4096, 121, 12.0), (1025, 4096, 121, 12.0)])
def test_e4m3(T, H, shift, size, dtype):
    """5-bit odd numbers in every binade, half way between two of 4 bits, and odd multiples of
    half the smallest step; a largest value of 256 in each block makes its scale 1. The same at
    the smallest scale, and past the range of fp32 (there one block, the others zeros)."""
    cases, steps = [256.0], {256.0: 0.0}
    for j in range(-10, 5):
        for y in range(17 if j > -10 else 1, 32 if j < 4 else 28, 2):
            cases.append(y * 2.0 ** j)
            steps[cases[-1]] = 2.0 ** j
    cases.append(256.0)  # 128: a block each sign
    assert len(cases) == 128
    unit = 2.0 ** shift
    cases = [(y * unit, size, y * unit * 3 / size) for y in cases]
    if shift > 0:
        cases += [(0.0, 0.0, 0.0)] * (H - 128)
    t, w, m = row(cases, H, dtype)
    step = torch.tensor([steps.get(v, 0.0) for v in (m.abs() / unit).tolist()], dtype=torch.float64) * unit
    for off in OFFS:
        q, scale = norm(t, w, off, T, dtype, q_dtype=torch.float8_e4m3fn)[2:]
        assert (scale[:, 0] == unit).all() and ((scale == unit) | (scale == 1)).all()
        want = m + m.sign() * (step if off > 0 else -step)
        got = q.double().cpu() * scale.double().cpu().repeat_interleave(128, 1)
        bad = (got != want).any(0).nonzero().flatten().tolist()
        assert not bad, f"{off}: {len(bad)} of {H} columns: {[(float(m[i]), float(got[0, i])) for i in bad[:4]]}"
