"""The 8-bit products at the ends of the scales' range: the product of a row's and a
weight block's scale is formed first, in fp32. It may come up to the largest finite value,
with any sign; below 2^-126 it is rounded to whole steps of 2^-149, which costs a result
at most 2^-150 of the sum of |a w| (the values as stored, without scales)."""
import pytest
import torch

import combine_moe_route_03_amd as moe
from fp8_reference import F32_STEP, RUN8
from test_gpu_fp8 import DEV, F8, gen

pytestmark = pytest.mark.gpu
N = 144
# one K step, streamed and tiled
SIZES = [(3, 128), (20, 384), (300, 256), (290, 640)]


def product(a, sa, w, sw):
    """The kernel's result on one expert, and (exact, |a| |w| per block) in 64 bits."""
    rows, K = a.shape
    out = moe.expert_gemm_fp8(a.to(DEV), sa.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV),
                              torch.full((1,), rows, dtype=torch.int32, device=DEV), w.to(DEV), sw.to(DEV))
    ad, wd = a.float().double(), w[0].float().double()
    want, mag, raw = (torch.zeros(rows, N, dtype=torch.float64) for _ in range(3))
    s_of = sw[0].double().repeat_interleave(128, 0)[:N]
    for b in range(K // 128):
        j = slice(128 * b, 128 * b + 128)
        s = sa[:, b].double()[:, None] * s_of[:, b][None]
        m = ad[:, j].abs() @ wd[:, j].abs().t()
        want += s * (ad[:, j] @ wd[:, j].t())
        mag += s.abs() * m
        raw += m
    return out.cpu().double(), want, mag, raw


def check(got, want, mag, raw, K):
    acc = ((K + 3 * (K // 128 + 1)) * F32_STEP + RUN8) * mag + 2.0 ** -150 * raw
    # the rounding to bf16 (below its normal range to half of 2^-133), and a step of fp32
    # subnormals for each of the sum's terms
    acc = acc + K // 128 * 2.0 ** -149
    bound = acc + 2.0 ** -8 * (want.abs() + acc) + 2.0 ** -134
    assert bool(torch.isfinite(got).all())
    assert float(((got - want).abs() - bound).max()) <= 0


def signs(*shape, seed):
    return torch.randint(0, 2, shape, generator=gen(seed)).float() * 2 - 1


@pytest.mark.parametrize("rows,K", SIZES)
def test_largest(rows, K):
    """Scale products just below 2^128, of either sign, on the smallest e4m3 values
    (products 2^-18), with rows and weight blocks of zeros."""
    print(f"[scales] largest rows={rows} K={K}", flush=True)
    a = signs(rows, K, seed=1) * 2.0 ** -9
    w = signs(1, N, K, seed=2) * 2.0 ** -9
    a[1::3] = 0
    w[:, 128:] = 0
    e = torch.randint(0, 100, (K // 128,), generator=gen(3)).double()
    sa = (signs(rows, K // 128, seed=4).double() * torch.exp2(e)).float()
    sw = (torch.exp2(127 - e) * (2 - 2.0 ** -20)).float().expand(1, 2, -1).contiguous()
    sw[:, 1] *= -1
    got, want, mag, raw = product(a.to(F8), sa, w.to(F8), sw)
    assert float(mag.max()) > 2.0 ** 115
    assert not bool(got[1::3].any()) and not bool(got[:, 128:].any())
    check(got, want, mag, raw, K)


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("top", [-126, -138, -149, -160])
def test_smallest(rows, K, top):
    """Scale products from below fp32's normal range to nothing, on the largest values."""
    print(f"[scales] smallest rows={rows} K={K} 2^{top}", flush=True)
    a, w = signs(rows, K, seed=1) * 448, signs(1, N, K, seed=2) * 448
    e = torch.randint(60, 100, (K // 128,), generator=gen(3)).double()
    frac = torch.rand(rows, K // 128, generator=gen(4)).double() + 1
    sa = (frac * torch.exp2(-e + 20)).float()
    sw = (torch.exp2(e - 20 + top) * 1.37).float().expand(1, 2, -1).contiguous()
    assert float(sw.min()) > 2.0 ** -126 and float(sa.min()) > 2.0 ** -126
    got, want, mag, raw = product(a.to(F8), sa, w.to(F8), sw)
    check(got, want, mag, raw, K)


@pytest.mark.parametrize("rows,K", SIZES)
def test_opposite(rows, K):
    """Scales at opposite ends whose product is ordinary, and scales of zero."""
    a, w = signs(rows, K, seed=1), signs(1, N, K, seed=2)
    sa = torch.full((rows, K // 128), 1.25 * 2.0 ** 126)
    sa[::5] = 0
    sw = torch.full((1, 2, K // 128), -1.5 * 2.0 ** -126)
    sw[:, 1] = 0
    got, want, mag, raw = product(a.to(F8), sa, w.to(F8), sw)
    assert not bool(got[::5].any()) and not bool(got[:, 128:].any())
    check(got, want, mag, raw, K)
