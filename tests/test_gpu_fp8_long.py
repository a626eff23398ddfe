"""The 8-bit products and FFN with more K steps than the streamed kernel keeps scales of
at a time (64), in either product, and with nearly all rows on one expert of many."""
import pytest

import test_gpu_fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,H,I", [
    ([5, 0, 30], 8320, 128), ([9], 16512, 128), ([300, 2], 8320, 128), ([5, 33], 128, 8320),
    ([300], 256, 8320)])
def test_ffn(counts, H, I):
    test_gpu_fp8.test_expert_swiglu_fp8(counts, H, I)


@pytest.mark.parametrize("counts,gap,N,K", [
    ([1200] + [0] * 40 + [1, 7], 1, 272, 384), ([0] * 99 + [2500], 0, 144, 256), ([7, 12], 3, 64, 16640)])
def test_product(counts, gap, N, K):
    test_gpu_fp8.test_expert_gemm_fp8(counts, gap, N, K)


@pytest.mark.parametrize("counts", [[1500] + [0] * 60, [3, 1300, 0, 2] * 13 + [0] * 600])
def test_ffn_of_one_long_expert(counts):
    """Streamed for its mean, in many row tiles of one expert."""
    assert sum(counts) <= 28 * len(counts)
    test_gpu_fp8.test_expert_swiglu_fp8(counts, 128, 128)
