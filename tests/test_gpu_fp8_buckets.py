"""Buckets of the 8-bit products that do not lie in [0, rows): they give no output,
not even for the rows of theirs that do lie there, and the others' outputs are what
they are without them, however many rows the bad ones claim."""
import pytest
import torch

import combine_moe_route_03_amd as moe
from test_gpu_fp8 import DEV, fp8_weights, randn

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def with_bad_buckets(rows):
    """(offsets, counts) of eight experts: the fifth and the last lie in the rows, [3, 40)
    and [40, rows - 5); the others leave them."""
    offs = [rows + 5, -1, 1, rows - 50, 3, 2 ** 31 - 1, 0, 40]
    cnts = [rows, rows, rows, 100, 37, rows, rows + 1, rows - 45]
    return i32(offs), i32(cnts)


def without(cnts):
    keep = i32([0, 0, 0, 0, 1, 0, 0, 1])
    return cnts * keep


# streamed (few rows an expert; one K step) and tiled, with many column tiles
@pytest.mark.parametrize("rows,N,K", [(200, 2048, 256), (1500, 1024, 128), (1500, 512, 384),
                                      (3000, 2048, 256)])
def test_product(rows, N, K):
    print(f"[bad buckets] product rows={rows} N={N} K={K}", flush=True)
    a, sa = moe.quantize(randn(rows, K, seed=1).to(DEV))
    w, sw = [t.to(DEV) for t in fp8_weights(8, N, K, 2)]
    offs, cnts = with_bad_buckets(rows)
    want = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_gemm_fp8(a, sa, offs, without(cnts), w, sw, out=want)
    assert bool((want[:3] == 3).all()) and bool((want[-5:] == 3).all())
    assert not bool((want[3:-5] == 3).all(1).any())
    out = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_gemm_fp8(a, sa, offs, cnts, w, sw, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("rows", [40, 600])
@pytest.mark.parametrize("bad", [(-5, 20), (10, 3000), (35, 1 << 30), (1, None)])
def test_a_bucket_partly_in_the_rows(rows, bad):
    """One bucket alone, some tiles of which lie in the rows."""
    off, cnt = bad[0], bad[1] or rows
    a, sa = moe.quantize(randn(rows, 256, seed=1).to(DEV))
    w, sw = [t.to(DEV) for t in fp8_weights(1, 64, 256, 2)]
    out = torch.full((rows, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_gemm_fp8(a, sa, i32([off]), i32([cnt]), w, sw, out=out)
    assert bool((out == 3).all())


@pytest.mark.parametrize("rows,H,I", [(200, 1024, 512), (1500, 512, 256)])
def test_ffn(rows, H, I):
    print(f"[bad buckets] ffn rows={rows} H={H} I={I}", flush=True)
    a, sa = moe.quantize(randn(rows, H, seed=1).to(DEV))
    wg, sg = [t.to(DEV) for t in fp8_weights(8, 2 * I, H, 2)]
    wd, sd = [t.to(DEV) for t in fp8_weights(8, H, I, 4)]
    shape = moe.Shape(rows, H, 8, 1, 1, 1, torch.bfloat16)
    offs, cnts = with_bad_buckets(rows)
    got = []
    for c in (cnts, without(cnts)):
        ws = torch.zeros(moe.expert_swiglu_fp8_workspace_bytes(shape, I), dtype=torch.uint8, device=DEV)
        out = torch.full((rows, H), 3.0, dtype=torch.bfloat16, device=DEV)
        moe.expert_swiglu_fp8(a, sa, offs, c, shape, wg, sg, wd, sd, expert_out=out, workspace=ws)
        got.append((out, ws))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert not bool((got[0][0][3:-5] == 3).all(1).any())
