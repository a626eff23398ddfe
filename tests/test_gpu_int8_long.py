"""Rows, weights and results of the integer path and the norm past 2^31 bytes, where a
32-bit offset would wrap: the last rows against the reference."""
import pytest
import torch

import combine_moe_route_03_amd as moe
import int8_reference as ref
from test_gpu_int8 import DEV, I32, buckets, ints, scales
from test_gpu_norm import BF16, check_norm, hidden

pytestmark = pytest.mark.gpu


def test_quantize_and_norm():
    T, H = 33000, 65536
    x = torch.zeros(T, H, device=DEV, dtype=BF16)
    x[-9:] = hidden(9, H, BF16, 1)
    q, scale = moe.quantize_int8(x)
    want_q, want_s = ref.int8_rows(x[-9:])
    assert torch.equal(q[-9:].double(), want_q) and torch.equal(scale[-9:].double(), want_s)
    assert int(q[:100].abs().max()) == 0 and (scale[:-9] == 1).all()
    w = (1 + 0.3 * torch.randn(H, device=DEV)).to(BF16)
    got = moe.add_rms_norm(x, w, 1e-6, residual=x, q_dtype=torch.int8, q=q, scale=scale)
    check_norm(x[-9:], w, 1e-6, x[-9:], torch.int8, tuple(v[-9:] for v in got))


@pytest.mark.parametrize("rows,N,K", [(270001, 4112, 8192), (270001, 4112, 272)])
def test_tiled(rows, N, K):
    a, sa = ints(rows, K, seed=1), scales(rows, seed=2)
    w, sw = ints(1, N, K, seed=3), scales(1, N, seed=4)
    offs, cnts, _ = buckets([rows])
    out = moe.expert_gemm_int8(a, sa, offs, cnts, w, sw)
    want = ref.scaled_sums(a[-300:], sa[-300:], w[0], sw[0]).to(BF16)
    assert torch.equal(out[-300:], want)


def test_streamed_rows():
    """Few rows an expert, the last ones past 2^31 bytes of rows."""
    E, N, K, rows = 1024, 16, 96000, 24000
    a, sa = ints(rows, K, seed=1), scales(rows, seed=2)
    w, sw = ints(E, N, K, seed=3), scales(E, N, seed=4)
    counts = [23] * E
    counts[-1] = rows - 23 * (E - 1)
    offs, cnts, total = buckets(counts)
    assert total == rows
    out = moe.expert_gemm_int8(a, sa, offs, cnts, w, sw)
    n = counts[-1]
    assert torch.equal(out[-n:], ref.scaled_sums(a[-n:], sa[-n:], w[-1], sw[-1]).to(BF16))


@pytest.mark.parametrize("each", [3, 60])
def test_weights(each):
    """The last experts' weights past 2^31 bytes."""
    E, N, K = 300, 2064, 4096
    rows = E * each
    a, sa = ints(rows, K, seed=1), scales(rows, seed=2)
    w, sw = ints(E, N, K, seed=3), scales(E, N, seed=4)
    offs, cnts, _ = buckets([each] * E)
    index = torch.arange(rows - 1, -1, -1, **I32)
    out = moe.expert_gemm_int8(a, sa, offs, cnts, w, sw, row_token=index)
    b, sb = a.flip(0), sa.flip(0)
    for e in (0, 1, E - 2, E - 1):
        r = slice(e * each, (e + 1) * each)
        assert torch.equal(out[r], ref.scaled_sums(b[r], sb[r], w[e], sw[e]).to(BF16))
