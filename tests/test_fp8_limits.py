"""Sizes at the limits of the 8-bit entry points, on the CPU: what a kernel cannot count
is refused. Calls whose sizes pass fail at a later check (a misaligned pointer, a
workspace of no bytes), so that none launches."""
import ctypes

import pytest

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
