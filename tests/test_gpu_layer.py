"""The small MoE layer (routing, experts, combine from logits to y) on the GPU
against its definition in 64 bits, within the bounds of fp8_reference.layer."""
import numpy as np
import pytest
import torch

import combine_moe_route_03_amd as moe
import fp8_reference as ref
from test_gpu_fp8 import DEV, fp8_weights, randn

pytestmark = pytest.mark.gpu

# T, H, E, k, I, routing
CASES = [
    (1, 128, 1, 1, 128, "iid"), (1, 512, 8, 8, 256, "iid"), (1, 256, 300, 5, 128, "iid"),
    (2, 128, 16, 2, 384, "iid"), (4, 256, 64, 32, 128, "iid"), (4, 128, 1000, 4, 128, "iid"),
    (5, 256, 12, 3, 128, "ties"), (17, 384, 64, 6, 256, "iid"), (16, 128, 4, 4, 128, "iid"),
    (33, 128, 40, 1, 128, "one"), (64, 256, 1024, 16, 128, "iid"), (128, 128, 24, 8, 128, "hot"),
    (128, 128, 1, 1, 128, "iid"), (127, 256, 9, 2, 128, "one"), (31, 128, 1024, 32, 128, "iid"),
    (3, 1408, 6, 2, 128, "masked"),
]


def logits_of(T, E, k, routing, seed=5):
    l = randn(T, E, seed=seed)
    if routing == "ties":
        return torch.randint(-1, 2, (T, E), generator=torch.Generator().manual_seed(seed)).float()
    if routing == "one":  # one expert takes a pick of every token
        l[:, E // 2] += 50
    if routing == "hot":
        l[:, : k // 2] += 20
    if routing == "masked":  # experts masked by the type's lowest value
        l[:, k:] = torch.finfo(torch.float32).min
    return l


def weights(E, H, I, fp8, seed=7):
    if fp8:
        (wg, sg), (wd, sd) = fp8_weights(E, 2 * I, H, seed), fp8_weights(E, H, I, seed + 3)
        return (wg, wd, sg, sd), ref.dequantize(wg, sg, 128), ref.dequantize(wd, sd, 128)
    wg = randn(E, 2 * I, H, seed=seed, scale=0.05).to(torch.bfloat16)
    wd = randn(E, H, I, seed=seed + 1, scale=0.05).to(torch.bfloat16)
    return (wg, wd, None, None), wg.double(), wd.double()


def call(logits, x, k, w, **kw):
    wg, wd, sg, sd = [None if t is None else t.to(DEV) for t in w]
    return moe.layer(logits.to(DEV), x.to(DEV), k, wg, wd, s_gate_up=sg, s_down=sd, **kw)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,E,k,I,routing", CASES)
def test_layer(T, H, E, k, I, routing, fp8):
    if not fp8 and I == 128:
        I = 192 if H % 256 else 64  # half blocks are allowed with 16-bit weights
    print(f"[layer] T={T} H={H} E={E} k={k} I={I} {routing} fp8={fp8}", flush=True)
    logits = logits_of(T, E, k, routing)
    x = randn(T, H, seed=6).to(torch.bfloat16)
    w, wg, wd = weights(E, H, I, fp8)
    y, idx, gate = call(logits, x, k, w)
    ridx, rgate, ry, bound = ref.layer(logits.double(), x.double(), k, wg, wd)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    rel = np.abs(gate.cpu().double().numpy() - rgate)
    assert (rel <= 2.0 ** -24 * rgate + 1e-15 * rgate + 2.0 ** -150).all()  # evaluated in double, rounded once
    err = (y.cpu().double() - ry).abs() - bound
    assert float(err.max()) <= 0, f"{float(err.max())} over the bound"


# Experts with more picks than one group of 32, through every shape of the down kernel: 8 or
# 16 columns a block, 8 or 16 waves; two, three and four groups.
GROUPS = [(50, 128, 5, 2, 256, "one"), (100, 128, 3, 2, 128, "one"), (96, 256, 70, 4, 128, "hot"),
          (128, 256, 5, 3, 384, "hot"), (40, 4096, 2, 1, 128, "one"), (70, 4096, 1, 1, 128, "iid"),
          (128, 4096, 3, 2, 256, "one"), (128, 4096, 40, 2, 128, "hot")]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,E,k,I,routing", GROUPS)
def test_layer_many_picks_an_expert(T, H, E, k, I, routing, fp8):
    test_layer(T, H, E, k, I, routing, fp8)


def test_layer_agrees_with_the_separate_steps():
    """moe_route, moe_dispatch, moe_expert_swiglu and moe_combine on the same
    inputs: the same picks and weights bit for bit; y differs by the rounding of
    the experts' outputs (2^-8 of each) and of y on either side."""
    T, H, E, k, I = 21, 256, 16, 4, 192
    logits = logits_of(T, E, k, "iid")
    x = randn(T, H, seed=6).to(torch.bfloat16)
    w, wg, wd = weights(E, H, I, False)
    y, idx, gate = call(logits, x, k, w)
    shape = moe.Shape(T, H, E, k, 1, 1, torch.bfloat16)
    i2, g2 = moe.route(logits.to(DEV), k)
    d = moe.dispatch(x.to(DEV), i2, E, 1, 1)
    eo = moe.expert_swiglu(d["send_buf"], d["expert_offsets"], d["expert_counts"], shape,
                           w[0].to(DEV), w[1].to(DEV))
    y2 = moe.combine(eo, g2, d["pos"], shape)
    assert torch.equal(idx, i2) and torch.equal(gate, g2)
    _, _, ry, bound = ref.layer(logits.double(), x.double(), k, wg, wd)
    # the separate steps round each expert's output too: 2^-8 of sum w |o|
    o = eo.float()[d["pos"].long().view(-1)].view(T, k, H)
    extra = 2.0 ** -8 * (g2.unsqueeze(-1) * o.abs()).sum(1).cpu().double()
    assert float(((y.cpu() - y2.cpu()).double().abs() - 2 * bound - extra).max()) <= 0


def test_layer_zero_tokens():
    w, _, _ = weights(4, 128, 128, False)
    y, idx, gate = call(torch.empty(0, 4), torch.empty(0, 128, dtype=torch.bfloat16), 2, w)
    assert y.shape == (0, 128) and idx.shape == (0, 2)


@pytest.mark.parametrize("T", [3, 40])
def test_layer_weights_past_32_bits(T):
    """A token's experts lie more than 2^32 bytes into the weights: y is that of a layer
    of these experts alone."""
    E, H, I, k, n = 200, 4096, 1408, 4, 8
    g = torch.Generator(DEV).manual_seed(9)
    wg, wd = [torch.empty(s, dtype=torch.bfloat16, device=DEV).normal_(std=0.05, generator=g)
              for s in ((E, 2 * I, H), (E, H, I))]
    logits = torch.randn(T, E, device=DEV, generator=g)
    logits[:, -n:] += 50
    x = randn(T, H, seed=6).to(torch.bfloat16).to(DEV)
    y, idx, gate = moe.layer(logits, x, k, wg, wd)
    y1, idx1, gate1 = moe.layer(logits[:, -n:].contiguous(), x, k, wg[-n:], wd[-n:])
    assert torch.equal(idx, idx1 + E - n) and torch.equal(gate, gate1)
    assert torch.equal(y, y1) and bool(y.float().norm() > 0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [4, 60, 128])
def test_layer_nan_stays_in_its_token(T, fp8):
    H, E, k, I = 256, 6, 3, 128
    w, _, _ = weights(E, H, I, fp8)
    logits, x = logits_of(T, E, k, "iid"), randn(T, H, seed=6).to(torch.bfloat16)
    clean, _, _ = call(logits, x, k, w)
    x[T // 2, 7] = float("nan")
    y, _, _ = call(logits, x, k, w)
    keep = torch.arange(T, device=DEV) != T // 2
    assert bool(y[T // 2].isnan().all()) and torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_layer_repeats_streams_and_graphs(T, fp8):
    """The same bits from every call (the sums have a fixed order), on another
    stream, and from two captured graphs with a workspace each, replayed in turn
    with eager work between."""
    H, E, k, I = 256, 24, 4, 128
    w, _, _ = weights(E, H, I, fp8)
    wg, wd, sg, sd = [None if t is None else t.to(DEV) for t in w]
    shape = moe.Shape(T, H, E, k, 1, 1, torch.bfloat16)
    nbytes = moe.layer_workspace_bytes(shape, I)
    ins = [(logits_of(T, E, k, "iid", seed=s).to(DEV), randn(T, H, seed=s).to(torch.bfloat16).to(DEV))
           for s in (1, 2)]

    def bufs():
        return dict(topk_idx=torch.empty(T, k, dtype=torch.int32, device=DEV),
                    topk_w=torch.empty(T, k, device=DEV),
                    y=torch.empty(T, H, dtype=torch.bfloat16, device=DEV),
                    workspace=torch.empty(nbytes, dtype=torch.uint8, device=DEV).fill_(0xA5))

    def step(i, b):
        moe.layer(*ins[i], k, wg, wd, s_gate_up=sg, s_down=sd, **b)

    want = []
    for i in range(2):
        b = bufs()
        step(i, b)
        torch.cuda.synchronize()
        want.append(b["y"].clone())
        for _ in range(4):
            step(i, b)
            torch.cuda.synchronize()
            assert torch.equal(b["y"], want[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = bufs()
    with torch.cuda.stream(side):
        step(0, b)
    torch.cuda.synchronize()
    assert torch.equal(b["y"], want[0])
    graphs = []
    for i in range(2):
        b = bufs()
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(i, b)
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                step(i, b)
        graphs.append((g, b))
    eager = bufs()
    for rep in range(3):
        for (g, b), v in zip(graphs, want):
            b["y"].fill_(9.0)
            b["workspace"].fill_(0x5A)
            step(rep % 2, eager)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(b["y"], v), rep
