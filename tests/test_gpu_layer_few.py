"""The layer of up to 8 tokens, and of rows of 4096 and more, through every form of its
two kernels, against the definition in 64 bits within the bounds of
fp8_reference.layer.

Gate/up has two waves a unit while min(T k, E) * I / 8 < 4096, one from there on, and
other routing registers for more than 256 experts. Down has 8 columns a block below
H = 4096, 16 from there on; each of its 16 waves walks a run of experts."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
from test_gpu_fp8 import randn
from test_gpu_layer import call, logits_of, weights

pytestmark = pytest.mark.gpu

# T, H, E, k, I, routing
TWO_WAVES = [(8, 128, 63, 8, 512, "iid"), (8, 128, 300, 7, 512, "iid"), (4, 256, 7, 7, 1408, "iid"),
             (7, 128, 300, 1, 256, "one")]
ONE_WAVE = [(8, 128, 64, 8, 512, "iid"), (8, 128, 300, 8, 512, "iid"), (3, 256, 30, 8, 1408, "iid"),
            (5, 128, 1024, 32, 256, "iid"), (8, 256, 256, 4, 1024, "ties"), (8, 384, 257, 4, 1152, "iid"),
            (8, 128, 70, 8, 768, "hot"), (7, 128, 300, 6, 1408, "one")]
WIDE = [(1, 4096, 1, 1, 128, "iid"), (1, 4096, 8, 8, 128, "iid"), (8, 4096, 40, 6, 128, "iid"),
        (5, 4096, 24, 4, 256, "hot"), (2, 4224, 3, 2, 384, "iid"), (6, 4096, 300, 8, 128, "iid"),
        (3, 7168, 20, 8, 128, "iid"), (8, 4096, 1, 1, 1408, "iid"), (7, 4608, 18, 3, 256, "one"),
        (20, 7168, 8, 2, 128, "iid"), (128, 4224, 6, 2, 128, "hot")]


def waves(T, E, k, I):
    return 1 if min(T * k, E) * (I // 8) >= 4096 else 2


def run(T, H, E, k, I, routing, fp8):
    print(f"[layer few] T={T} H={H} E={E} k={k} I={I} {routing} fp8={fp8}", flush=True)
    logits = logits_of(T, E, k, routing)
    x = randn(T, H, seed=6).to(torch.bfloat16)
    w, wg, wd = weights(E, H, I, fp8)
    y, idx, gate = call(logits, x, k, w)
    ridx, rgate, ry, bound = ref.layer(logits.double(), x.double(), k, wg, wd)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    rel = np.abs(gate.cpu().double().numpy() - rgate)
    assert (rel <= 2.0 ** -24 * rgate + 1e-15 * rgate + 2.0 ** -150).all()
    err = (y.cpu().double() - ry).abs() - bound
    assert float(err.max()) <= 0, f"{float(err.max())} over the bound"
    again, _, _ = call(logits, x, k, w)
    assert torch.equal(y, again)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,E,k,I,routing", TWO_WAVES)
def test_two_waves_a_unit(T, H, E, k, I, routing, fp8):
    assert waves(T, E, k, I) == 2
    run(T, H, E, k, I, routing, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,E,k,I,routing", ONE_WAVE)
def test_one_wave_a_unit(T, H, E, k, I, routing, fp8):
    assert waves(T, E, k, I) == 1
    run(T, H, E, k, I, routing, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,E,k,I,routing", WIDE)
def test_wide_rows(T, H, E, k, I, routing, fp8):
    run(T, H, E, k, I, routing, fp8)


@pytest.mark.parametrize("T", [1, 8])
def test_wide_rows_half_blocks(T):
    """16-bit weights with I a multiple of 64 only."""
    run(T, 4096, 20, 4, 64, "iid", False)
    run(T, 4096, 20, 4, 192, "iid", False)
