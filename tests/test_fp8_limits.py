"""Sizes at the limits of the 8-bit entry points, on the CPU: what a kernel cannot count
is refused, and nothing is cut to 32 bits on the way. Calls whose sizes pass fail at a later check (a misaligned pointer, a
workspace of no bytes), so that none launches."""
import ctypes

import pytest
import torch

import combine_moe_route_03_amd as moe
from test_abi import ALIGN, ARG, FAKE, WORKSPACE, _shape

ODD16 = ctypes.c_void_p((1 << 20) + 8)


def gemm(rows, E, N, K):
    return moe.lib().moe_expert_gemm_fp8(rows, E, N, K, *(FAKE,) * 6, ODD16, None)


def ffn(T, E, H, I):
    sh = _shape(T=T, k=1, E=E, H=H, R=1, W=1)
    return moe.lib().moe_expert_swiglu_fp8(ctypes.byref(sh), I, *(FAKE,) * 10, 0, None)


def stream_threads(rows, E, N):
    """A block of 512 threads for each tile of 32 rows and 256 columns."""
    return (rows // 32 + min(rows, E)) * -(-N // 256) * 512


@pytest.mark.parametrize("E,N,K", [(1024, (1 << 22) - 16, 256), (1023, (1 << 22) - 16, 256),
                                   (512, (1 << 22) - 16, 512), (1024, 1 << 21, 384)])
def test_streamed_grids_beyond_32_bits_are_refused(E, N, K):
    """At up to 28 rows an expert whatever K is; with one more the weights are not streamed."""
    rows = 28 * E
    assert stream_threads(rows, E, N) >= 1 << 32 and E * N * K < 1 << 40
    assert gemm(rows, E, N, K) == ARG
    assert gemm(rows + 1, E, N, K) == ALIGN


def test_streamed_grids_within_32_bits_are_taken():
    E, N = 512, 1 << 21
    assert (1 << 31) < stream_threads(28 * E, E, N) < (1 << 32) - 512 * 64
    assert gemm(28 * E, E, N, 256) == ALIGN


def test_ffn_grids_beyond_32_bits_are_refused():
    """The same for the FFN's gate/up product (rows 2 I of weights)."""
    E, H, I = 600, 256, (1 << 21) - 128
    assert stream_threads(28 * E, E, 2 * I) >= 1 << 32 and E * 2 * I * H < 1 << 40
    assert ffn(28 * E, E, H, I) == ARG
    assert ffn(28 * E + 1, E, H, I) == WORKSPACE


def test_dispatch_limits():
    for dtype, most in ((moe.MOE_BF16, 1 << 27), (moe.MOE_F32, 1 << 26)):
        for T, H, st in ((most - 1, 16, ALIGN), (most, 16, ARG), (most // 2, 144, ARG)):
            sh = _shape(T=T, k=1, E=4, H=H, R=1, W=1, dtype=dtype)
            got = moe.lib().moe_dispatch_copy_fp8(ctypes.byref(sh), FAKE, FAKE, ODD16, FAKE, None)
            assert got == st, (dtype, T, H)


@pytest.mark.parametrize("E,H,I", [
    (1, 128, (1 << 20) - 64), (1, 128, 1 << 20), (1, (1 << 23) - 128, 64), (1, 1 << 23, 64),
    (1, 512, (1 << 20) - 64), (1, 1024, 1 << 19), (1, 1024, (1 << 19) - 64), (1024, 1024, 1 << 18),
    (1023, 1024, (1 << 19) - 64), (1024, 1024, (1 << 19) - 64), (1024, 1152, (1 << 19) - 64), (1, 128, 32)])
def test_layer_limits(E, H, I):
    """What the header says of I and H is what is taken."""
    within = I % 64 == 0 and I < 1 << 20 and H < 1 << 23 and 4 * I * H < 1 << 31 \
        and 2 * E * I * H < 1 << 40
    sh = _shape(T=128, k=1, E=E, H=H, R=1, W=1)
    assert (moe.lib().moe_layer_workspace_bytes(ctypes.byref(sh), I) > 0) == within


# ------------------------------------------------------------ sizes past 32 bits

BIG = (1 << 32) + 5  # what ctypes would cut to 5
F8, BF16, F32, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32


def meta(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("shape", [(BIG, 16), (1 << 16, (1 << 16) + 1, 1, 16), (1, BIG // 16 * 16)])
def test_quantize_of_more_than_32_bits_of_rows(shape):
    """The rows, their batches together or the columns."""
    for block_rows in (1, 128):
        with pytest.raises(ValueError, match="32 bits"):
            moe.quantize(meta(*shape), block_rows=block_rows)


def test_shapes_of_more_than_32_bits():
    for name in "THEkRW":
        kw = dict(T=4, H=128, E=4, k=2, R=1, W=1, dtype=BF16)
        kw[name] = BIG
        with pytest.raises(ValueError, match="32 bits"):
            moe.Shape(**kw)


def test_products_and_layers_of_more_than_32_bits():
    s = moe.Shape(4, 128, 4, 2, 1, 1, BF16)
    i = meta(4, dtype=I32)
    for rows, E, N, K in ((BIG, 4, 64, 128), (8, 4, 1 << 33, 128), (8, 4, 64, 1 << 33)):
        with pytest.raises(ValueError, match="32 bits"):
            moe.expert_gemm_fp8(meta(rows, K, dtype=F8), meta(rows, K // 128, dtype=F32), i, i,
                                meta(E, N, K, dtype=F8), meta(E, -(-N // 128), K // 128, dtype=F32))
    I = 1 << 32
    wg, wd = meta(4, 2 * I, 128, dtype=F8), meta(4, 128, I, dtype=F8)
    sg, sd = meta(4, I // 64, 1, dtype=F32), meta(4, 1, I // 128, dtype=F32)
    with pytest.raises(ValueError, match="32 bits"):
        moe.expert_swiglu_fp8(meta(8, 128, dtype=F8), meta(8, 1, dtype=F32), i, i, s, wg, sg, wd, sd)
    for f in (moe.expert_swiglu_fp8_workspace_bytes, moe.layer_workspace_bytes):
        with pytest.raises(ValueError, match="32 bits"):
            f(s, I + 128)
    for T, k, inter in ((2, 1, I), (BIG, 1, 128), (0, BIG, 128)):
        with pytest.raises(ValueError, match="32 bits"):
            moe.layer(meta(T, 4, dtype=F32), meta(T, 128), k, meta(4, 2 * inter, 128), meta(4, 128, inter))
