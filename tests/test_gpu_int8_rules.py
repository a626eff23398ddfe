"""The grouped int8 product on both sides of the rules that choose its kernel: the same bits
from whichever is taken."""
import pytest
import torch

from test_gpu_int8 import buckets, check, ints, scales

pytestmark = pytest.mark.gpu


def stream_rows(K):
    """Rows an expert up to which the weights are streamed, as the library has it."""
    if K % 128:
        return 8
    return min(28, max(14, 14 + (K - 2816) * 14 // 1280))


@pytest.mark.parametrize("K", [2816, 2944, 3328, 3584, 3968, 4096, 4224, 3600])
def test_streamed_or_tiled_by_k(K):
    """A row more than the limit, the limit, a row less; experts of unlike sizes, the average so."""
    E, N = 12, 8208
    limit = stream_rows(K)
    w, sw = ints(E, N, K, seed=3), scales(E, N, seed=4)
    for rows in (limit * E - 1, limit * E, limit * E + 1):
        assert (rows + 16 * E) * N > 2 ** 20 + 16 * N  # not few results in all
        counts = [limit] * E
        counts[0] += 3
        counts[5] = limit - 3
        counts[-1] += rows - limit * E
        offs, cnts, total = buckets(counts)
        assert total == rows
        print(f"[rule] K={K} rows={rows}", flush=True)
        check(ints(rows, K, seed=1), scales(rows, seed=2), offs, cnts, w, sw)
