"""SiLU in the experts for the largest finite gates: silu(g) is g, or zero, up to the
largest fp32 value. Powers of two around one column, so every product, sum and
rounding is exact and the result is known."""
import pytest
import torch

import combine_moe_route_03_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# gate values over 2^127: 1.75 = 2.98e38 (of at most 3.40e38); u = 2^-120
GATES = [1.75, -1.75, 1.5, 1.0, -1.0, 0.875, -0.5, 2.0 ** -100, -2.0 ** -100]
WANT = [g * 2.0 ** 7 if g > 0 else 0.0 for g in GATES]  # silu(g) u


def expected(rows, H, scale=1.0):
    y = torch.zeros(rows, H)
    y[:, :len(WANT)] = torch.tensor(WANT) * scale
    return y


# one K step (streamed), few rows an expert (streamed), tiled
@pytest.mark.parametrize("rows,H", [(3, 128), (5, 256), (70, 256), (300, 512)])
def test_fp8_experts(rows, H):
    I = 128
    a = torch.zeros(rows, H)
    a[:, 0] = 1
    wg, wd = torch.zeros(1, 2 * I, H), torch.zeros(1, H, I)
    for j, g in enumerate(GATES):
        wg[0, j, 0] = g * 2 ** 8 if abs(g) > 2.0 ** -10 else 0
        wg[0, I + j, 0] = 1
        wd[0, j, j] = 1
    sg = torch.ones(1, 2, H // 128)
    sg[0, 0], sg[0, 1] = 2.0 ** 119, 2.0 ** -120
    f8 = torch.float8_e4m3fn
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device=DEV)
    shape = moe.Shape(rows, H, 1, 1, 1, 1, torch.bfloat16)
    out = moe.expert_swiglu_fp8(
        a.to(f8).to(DEV), torch.ones(rows, H // 128, device=DEV), i32(0), i32(rows), shape,
        wg.to(f8).to(DEV), sg.to(DEV), wd.to(f8).to(DEV),
        torch.ones(1, H // 128, 1, device=DEV))
    # h = 224, 192, 128, 112 and zeros: e4m3 values with the scale 2^-1
    want = expected(rows, H)
    want[:, [j for j, g in enumerate(GATES) if abs(g) < 2.0 ** -10]] = 0
    assert torch.equal(out.float().cpu(), want)


def bf16_weights(H, I):
    wg, wd = torch.zeros(1, 2 * I, H), torch.zeros(1, H, I)
    for j, g in enumerate(GATES):
        wg[0, j, 0] = g * 2.0 ** 127
        wg[0, I + j, 0] = 2.0 ** -120
        wd[0, j, j] = 1
    return wg.to(torch.bfloat16).to(DEV), wd.to(torch.bfloat16).to(DEV)


def bf16_rows(rows, H):
    x = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    return x


@pytest.mark.parametrize("T", [1, 7, 20, 128])
def test_layer(T):
    wg, wd = bf16_weights(256, 128)
    y, _, _ = moe.layer(torch.zeros(T, 1, device=DEV), bf16_rows(T, 256), 1, wg, wd)
    assert_exact(y, expected(T, 256))


@pytest.mark.parametrize("rows", [3, 300])
def test_bf16_experts(rows):
    H, I = 256, 128
    wg, wd = bf16_weights(H, I)
    shape = moe.Shape(rows, H, 1, 1, 1, 1, torch.bfloat16)
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device=DEV)
    out = moe.expert_swiglu(bf16_rows(rows, H), i32(0), i32(rows), shape, wg, wd)
    assert_exact(out, expected(rows, H))


def assert_exact(y, want):
    assert torch.equal(y.float().cpu(), want)
