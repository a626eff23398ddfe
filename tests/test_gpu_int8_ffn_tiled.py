"""The integer FFN through the tiled kernels of 256 and of 128 rows, gate/up and down: buckets of
uneven sizes, rows by index and in expert order, against 64 bits (int8_reference.py has the
bounds). The library's rule for the kernel is repeated here, so that a case says which one it
reaches."""
import pytest
import torch

import combine_moe_route_03_amd as moe
import int8_reference as ref
from test_gpu_int8 import DEV, I32, block_buffers, block_step, buckets, check_block, tiled

pytestmark = pytest.mark.gpu


def rows_of_a_tile(rows, E, N, K):
    """Rows of a tile of the kernel that a product takes; 0: streamed."""
    if not tiled(rows, E, N, K):
        return 0
    tiles = (rows + 64 * min(rows, E)) // 128 * ((N + 255) // 256)
    return 128 if K > 256 and (rows <= 128 * E or tiles <= 256) else 256


def uneven(E, rows, seed):
    """Counts of E experts that add up to rows: one with most of them, some with few, one none."""
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(E, generator=g) ** 2 + 0.02
    share[0] = 3.0
    counts = (share / share.sum() * rows).int().tolist()
    if E > 2:
        counts[2] = 0
    counts[min(1, E - 1)] += rows - sum(counts)
    return counts


# kernels of the two products, T * k rows; K steps on both sides of 16; inner columns that fill
# the last tile and that do not
CASES = [
    ((256, 128), 6000, 272, 3, 1040),    # 3 steps; 2 tiles of 256 columns and 16 more
    ((256, 256), 6000, 256, 4, 208),     # 2 steps of both products
    ((256, 256), 9000, 144, 1, 256),     # a part of a step, one expert
    ((256, 0), 5000, 208, 5, 128),       # rows that are no lines, a tile exactly
    ((256, 256), 10400, 2064, 2, 400),   # 17 steps, less than a round of tiles
    ((256, 256), 12000, 2064, 3, 1408),  # 17 steps, two rounds: long parts come last
    ((256, 256), 20001, 512, 7, 1040),   # 4 steps, more than two rounds: parts come first
    ((256, 256), 16384, 1936, 16, 880),  # 16 steps; short experts among long ones
    ((128, 128), 2500, 1040, 3, 880),
    ((128, 128), 4000, 4096, 40, 512),   # 32 steps, up to 128 rows an expert
]


def case(rows, H, E, I, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    offs, cnts, total = buckets(uneven(E, rows, seed))
    assert total == rows
    token = torch.randint(0, rows, (rows,), generator=g, device=DEV, dtype=torch.int32)
    x = torch.randn(rows, H, generator=g, device=DEV) * torch.exp(torch.randn(rows, 1, generator=g, device=DEV))
    # gates of a few units, where SiLU bends
    wg = torch.randn(E, 2 * I, H, generator=g, device=DEV) * H ** -0.5
    wd = torch.randn(E, H, I, generator=g, device=DEV) * I ** -0.5
    shape = moe.Shape(rows, H, E, 1, 1, 1, torch.bfloat16)
    return shape, offs, cnts, token, *moe.quantize_int8(x), *moe.quantize_int8(wg), *moe.quantize_int8(wd)


@pytest.mark.parametrize("kernels,rows,H,E,I", CASES)
def test_swiglu_tiled(kernels, rows, H, E, I):
    assert kernels == (rows_of_a_tile(rows, E, 2 * I, H), rows_of_a_tile(rows, E, H, I))
    shape, offs, cnts, token, x, sx, wg, sg, wd, sd = case(rows, H, E, I, seed=rows)
    out = moe.expert_swiglu_int8(x, sx, offs, cnts, shape, wg, sg, wd, sd, row_token=token)
    for e, (o, n) in enumerate(zip(offs.tolist(), cnts.tolist())):
        for a in range(o, o + n, 4096):  # bounds the 64-bit copies
            r = slice(a, min(a + 4096, o + n))
            t = token[r].long()
            want, bound = ref.swiglu(x[t], sx[t], wg[e], sg[e], wd[e], sd[e])
            over = float(((out[r].double() - want).abs() - bound).max())
            assert over <= 0, f"expert {e}, rows from {a}: {over} over the bound"
    t = token.long()
    rows_in_order = moe.expert_swiglu_int8(x[t], sx[t], offs, cnts, shape, wg, sg, wd, sd)
    assert torch.equal(rows_in_order, out)


@pytest.mark.parametrize("kernels,rows,H,E,I", [CASES[0], CASES[3], CASES[8]])
def test_swiglu_tiled_buckets(kernels, rows, H, E, I):
    """Gaps between the buckets, the last one first, indexes outside the tokens: rows outside the
    buckets stay, those of no token are zeros, the others have the bits they have without."""
    shape, offs, cnts, token, x, sx, wg, sg, wd, sd = case(rows, H, E, I, seed=rows + 1)
    want = moe.expert_swiglu_int8(x, sx, offs, cnts, shape, wg, sg, wd, sd, row_token=token)
    gap = 37
    total = rows + gap * E
    at, new = 0, [0] * E
    for e in reversed(range(E)):
        new[e], at = at, at + int(cnts[e]) + gap
    moved = torch.full((total,), -1, **I32)
    none = torch.zeros(total, dtype=torch.bool, device=DEV)
    live = torch.zeros(total, dtype=torch.bool, device=DEV)
    source = torch.zeros(total, dtype=torch.int64, device=DEV)
    for e in range(E):
        o, n = int(offs[e]), int(cnts[e])
        moved[new[e]:new[e] + n] = token[o:o + n]
        live[new[e]:new[e] + n] = True
        source[new[e]:new[e] + n] = torch.arange(o, o + n, device=DEV)
    for i, bad in enumerate((-1, total, 2 ** 31 - 1, -2 ** 31)):
        none[i::997] = True
        moved[i::997] = bad
    big = moe.Shape(total, H, E, 1, 1, 1, torch.bfloat16)
    xx = torch.cat([x, x[:total - rows]])
    ss = torch.cat([sx, sx[:total - rows]])
    out = torch.full((total, H), 9.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_swiglu_int8(xx, ss, torch.tensor(new, **I32), cnts, big, wg, sg, wd, sd, row_token=moved,
                           expert_out=out)
    assert kernels[0] == rows_of_a_tile(total, E, 2 * I, H)
    assert (out[~live] == 9).all() and (out[live & none] == 0).all()
    keep = live & ~none
    assert torch.equal(out[keep], want[source[keep]])


@pytest.mark.parametrize("T,H,E,k,I", [(3000, 512, 3, 2, 1040)])
def test_block_tiled(T, H, E, k, I):
    """A layer through the 256-row gate/up kernel, eager and captured, new inputs every replay."""
    assert rows_of_a_tile(T * k, E, 2 * I, H) == 256 and rows_of_a_tile(T * k, E, H, I) == 128
    b, other = block_buffers(T, H, E, k, I, seed=7), block_buffers(T, H, E, k, I, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block_step(b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    check_block(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block_step(b)
    for rep in range(3):
        b["x"].copy_(torch.randn(T, H, device=DEV))
        for name in ("total", "y", "eo", "out", "q", "s"):
            b[name].view(torch.uint8).fill_(0x5A)
        graph.replay()
        block_step(other)
        torch.cuda.synchronize()
        check_block(b)
        replayed = b["out"].clone()
        block_step(b)
        assert torch.equal(b["out"], replayed), rep
    check_block(other)
