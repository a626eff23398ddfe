"""What the 8-bit entry points and the small layer refuse, and the CPU side of
their reference. Nothing here launches a kernel."""
import ctypes

import numpy as np
import pytest
import torch

import combine_moe_route_03_amd as moe
import fp8_reference as ref
from test_abi import ALIGN, ARG, FAKE, OK, UNSUPPORTED, WORKSPACE, _shape

ODD4 = ctypes.c_void_p((1 << 20) + 2)
ODD16 = ctypes.c_void_p((1 << 20) + 8)


def test_reference_rounding_matches_torch():
    """round_e4m3 on every bf16 value up to 448 against torch's conversion."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[bits.float().abs() <= 448]
    assert np.array_equal(ref.round_e4m3(x.double().numpy()),
                          x.float().to(torch.float8_e4m3fn).float().double().numpy())


def test_reference_scales():
    """A block's maximum lands in (224, 448] after scaling, exactly at the ends."""
    for v, p in ((448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (1.75, -8), (1.0, -8), (2.0, -7)):
        x = np.zeros((1, 1, 128))
        x[0, 0, 5] = -v
        assert ref.quantize(x, 1)[1][0, 0, 0] == 2.0 ** p, v


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(batch=-1), ARG),
    (dict(rows=-1), ARG), (dict(cols=0), ARG), (dict(block_rows=64), ARG), (dict(block_rows=0), ARG),
    (dict(cols=24), ALIGN), (dict(rows=1 << 30, batch=4), ARG), (dict(rows=1 << 28), ARG),
    (dict(x=None), ARG), (dict(q=None), ARG), (dict(scale=None), ARG), (dict(x=ODD16), ALIGN),
    (dict(q=ODD16), ALIGN), (dict(scale=ODD4), ALIGN)])
def test_quantize_refusals(kw, status):
    a = dict(x=FAKE, dtype=1, batch=1, rows=4, cols=128, block_rows=1, q=FAKE, scale=FAKE)
    a.update(kw)
    assert moe.lib().moe_quantize(*a.values(), None) == status


def test_sizes_beyond_a_grid_are_refused():
    """Grids hold less than 2^32 threads: what would need more is refused, not half launched."""
    L = moe.lib()
    assert L.moe_quantize(FAKE, 1, 1 << 19, 1, 4096, 128, FAKE, FAKE, None) == ARG
    assert L.moe_quantize(FAKE, 1, 1 << 24, 1, 128, 128, FAKE, FAKE, None) == ARG
    args = (FAKE,) * 7 + (None,)
    assert L.moe_expert_gemm_fp8(1 << 24, 1, 4096, 128, *args) == ARG
    assert L.moe_expert_gemm_fp8(1 << 28, 1, 256, 128, *args) == ARG


def test_quantize_nothing():
    assert moe.lib().moe_quantize(None, 1, 0, 4, 128, 1, None, None, None) == OK
    assert moe.lib().moe_quantize(None, 0, 3, 0, 128, 128, None, None, None) == OK


def test_dispatch_copy_fp8_refusals():
    L = moe.lib()
    sh = _shape()

    def call(s, x=FAKE, pos=FAKE, q=FAKE, sc=FAKE):
        return L.moe_dispatch_copy_fp8(ctypes.byref(s) if s else None, x, pos, q, sc, None)

    assert call(None) == ARG
    assert call(_shape(H=24)) == ALIGN and call(_shape(dtype=2)) == UNSUPPORTED
    assert call(sh, x=None) == ARG and call(sh, q=None) == ARG and call(sh, sc=None) == ARG
    assert call(sh, pos=None) == ARG and call(sh, x=ODD16) == ALIGN and call(sh, q=ODD16) == ALIGN
    assert call(sh, pos=ODD4) == ALIGN and call(sh, sc=ODD4) == ALIGN


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), ARG), (dict(E=0), ARG), (dict(E=1025), ARG), (dict(N=8), ARG), (dict(N=24), ARG),
    (dict(K=64), ARG), (dict(K=192), ARG), (dict(N=1 << 20, K=1 << 12), ARG),
    (dict(K=1 << 23, N=16), ARG), (dict(N=1 << 22, K=128), ARG), (dict(a=None), ARG),
    (dict(sa=None), ARG), (dict(offs=None), ARG), (dict(cnts=None), ARG), (dict(w=None), ARG),
    (dict(sw=None), ARG), (dict(out=None), ARG), (dict(a=ODD16), ALIGN), (dict(w=ODD16), ALIGN),
    (dict(out=ODD16), ALIGN), (dict(sa=ODD4), ALIGN), (dict(sw=ODD4), ALIGN),
    (dict(offs=ODD4), ALIGN), (dict(cnts=ODD4), ALIGN)])
def test_expert_gemm_fp8_refusals(kw, status):
    a = dict(rows=8, E=4, N=64, K=128, a=FAKE, sa=FAKE, offs=FAKE, cnts=FAKE, w=FAKE, sw=FAKE,
             out=FAKE)
    a.update(kw)
    assert moe.lib().moe_expert_gemm_fp8(*a.values(), None) == status


def test_expert_gemm_fp8_without_rows():
    assert moe.lib().moe_expert_gemm_fp8(0, 4, 64, 128, None, None, FAKE, FAKE, FAKE, FAKE, None,
                                         None) == OK


def test_expert_swiglu_fp8_refusals():
    L = moe.lib()

    def call(I=128, ws=1 << 20, skip=None, odd=None, **kw):
        p = [FAKE] * 9 + [FAKE]
        if skip is not None:
            p[skip] = None
        if odd is not None:
            p[odd[0]] = odd[1]
        return L.moe_expert_swiglu_fp8(ctypes.byref(_shape(**kw)), I, *p, ws, None)

    need = L.moe_expert_swiglu_fp8_workspace_bytes(ctypes.byref(_shape()), 128)
    assert need == 64 * 2 * 128 + 64 * 2 * 4
    assert L.moe_expert_swiglu_fp8_workspace_bytes(ctypes.byref(_shape()), 192) == 0
    assert call(ws=need - 1) == WORKSPACE
    assert call(dtype=moe.MOE_F32) == UNSUPPORTED
    assert call(I=192) == ARG and call(I=0) == ARG and call(H=192) == ARG
    assert call(I=1 << 24, T=1, k=1) == ARG
    assert L.moe_expert_swiglu_fp8(None, 128, *[FAKE] * 10, 1 << 20, None) == ARG
    for i in range(10):
        assert call(skip=i) == ARG, i
    for i, p in ((0, ODD16), (1, ODD4), (2, ODD4), (3, ODD4), (4, ODD16), (5, ODD4), (6, ODD16),
                 (7, ODD4), (8, ODD16), (9, ODD16)):
        assert call(odd=(i, p)) == ALIGN, i


def test_layer_refusals():
    L = moe.lib()

    def call(I=128, wt=moe.MOE_F8E4M3, ws=1 << 24, skip=None, odd=None, **kw):
        p = [FAKE] * 10  # logits x wg sg wd sd idx w y workspace
        if skip is not None:
            p[skip] = None
        if odd is not None:
            p[odd[0]] = odd[1]
        return L.moe_layer(ctypes.byref(_shape(**kw)), I, wt, *p, ws, None)

    need = L.moe_layer_workspace_bytes(ctypes.byref(_shape()), 128)
    assert need >= 64 * 2 * 128 * 2
    assert call(ws=need - 1) == WORKSPACE
    assert call(T=129, k=1) == ARG and call(T=128, k=16, E=32) == ARG
    assert L.moe_layer_workspace_bytes(ctypes.byref(_shape(T=129, k=1)), 128) == 0
    assert call(I=192) == ARG and call(I=96, wt=moe.MOE_BF16) == ARG and call(H=192) == ARG
    assert call(wt=moe.MOE_F32) == UNSUPPORTED and call(dtype=moe.MOE_F32) == UNSUPPORTED
    for i in range(10):
        assert call(skip=i) == ARG, i
    assert call(wt=moe.MOE_BF16, skip=0) == ARG
    for i, p in ((0, ODD4), (1, ODD16), (2, ODD16), (3, ODD4), (4, ODD16), (5, ODD4), (6, ODD4),
                 (7, ODD4), (8, ODD16), (9, ODD16)):
        assert call(odd=(i, p)) == ALIGN, i


def test_binding_refusals():
    """Wrong types, shapes, strides and devices are refused before the library is called."""
    f8 = torch.float8_e4m3fn
    with pytest.raises(TypeError):
        moe.quantize(torch.zeros(4, 128, dtype=torch.float16))
    with pytest.raises(ValueError):
        moe.quantize(torch.zeros(4, 128), block_rows=32)
    with pytest.raises(ValueError):
        moe.quantize(torch.zeros(128))
    with pytest.raises(ValueError, match="contiguous"):
        moe.quantize(torch.zeros(128, 128).t())
    with pytest.raises(ValueError, match="current device"):
        moe.quantize(torch.zeros(4, 128))
    a, w = torch.zeros(4, 128, dtype=f8), torch.zeros(2, 64, 128, dtype=f8)
    i = torch.zeros(2, dtype=torch.int32)
    for bad in (dict(a=a.float()), dict(sa=torch.zeros(4, 2)), dict(w=w.float()),
                dict(o=i.long()), dict(sw=torch.zeros(2, 1, 2)), dict(c=i[:1])):
        g = dict(a=a, sa=torch.zeros(4, 1), o=i, c=i, w=w, sw=torch.zeros(2, 1, 1))
        g.update(bad)
        with pytest.raises((TypeError, ValueError)):
            moe.expert_gemm_fp8(*g.values())
    with pytest.raises(ValueError, match="s_gate_up"):
        moe.layer(torch.zeros(1, 2), torch.zeros(1, 128, dtype=torch.bfloat16), 1,
                  torch.zeros(2, 256, 128, dtype=f8), torch.zeros(2, 128, 128, dtype=f8))
