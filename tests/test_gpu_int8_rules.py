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


def one_round(rows, E, N):
    """Whether tiles of 128 rows by 256 columns are a round of the units, as the library has it."""
    return (rows + 64 * min(rows, E)) // 128 * ((N + 255) // 256) <= 256


@pytest.mark.parametrize("E,N,K,rows", [(1, 4112, 400, 1983), (1, 4112, 400, 1984), (1, 2048, 1024, 4159),
                                        (1, 2048, 1024, 4160), (7, 4096, 784, 1727), (7, 4096, 784, 1728),
                                        (12, 2816, 528, 2303), (12, 2816, 528, 2304)])
def test_tiles_of_128_or_256_rows(E, N, K, rows):
    assert rows > 128 * E and (rows + 16 * E) * N > 2 ** 20 + 16 * N
    assert one_round(rows, E, N) == (rows % 2 == 1) and one_round(rows - 1, E, N)
    counts = [rows // E] * E
    counts[0] += rows - sum(counts)
    if E > 3:
        counts[1], counts[2] = counts[1] + 129, counts[2] - 129
    offs, cnts, total = buckets(counts)
    assert total == rows
    print(f"[rule] E={E} N={N} K={K} rows={rows}", flush=True)
    check(ints(rows, K, seed=1), scales(rows, seed=2), offs, cnts, ints(E, N, K, seed=3), scales(E, N, seed=4))
