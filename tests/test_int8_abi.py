"""What the integer entry points and the norm refuse, and the CPU side of their
reference. Nothing here launches a kernel."""
import ctypes

import pytest
import torch

import combine_moe_route_03_amd as moe
import int8_reference as ref
from test_abi import ALIGN, ARG, FAKE, OK, UNSUPPORTED, WORKSPACE, _shape

ODD4 = ctypes.c_void_p((1 << 20) + 2)
ODD16 = ctypes.c_void_p((1 << 20) + 8)
OTHER = ctypes.c_void_p(1 << 21)


def test_reference_int8_rows():
    v = torch.tensor([[127.0, 0.5, 1.5, -2.5], [0, 0, 0, 0], [2.0 ** -140, 0, 0, 2.0 ** -127]])
    q, s = ref.int8_rows(v)
    assert q.tolist() == [[127, 0, 2, -2], [0, 0, 0, 0], [0, 0, 0, 0]]
    assert s.tolist() == [1.0, 1.0, 2.0 ** -126]
    ref.check_int8_rows(q.to(torch.int8), s, v)
    with pytest.raises(AssertionError):
        ref.check_int8_rows((q + 1).to(torch.int8), s, v)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(rows=-1), ARG),
    (dict(cols=0), ARG), (dict(cols=24), ALIGN), (dict(cols=65552), ARG), (dict(rows=1 << 27), ARG),
    (dict(rows=1 << 26, dtype=0), ARG), (dict(rows=1 << 26), ARG), (dict(rows=1 << 25, cols=144), ARG),
    (dict(x=None), ARG),
    (dict(q=None), ARG), (dict(scale=None), ARG), (dict(x=ODD16), ALIGN), (dict(q=ODD16), ALIGN),
    (dict(scale=ODD4), ALIGN)])
def test_quantize_int8_refusals(kw, status):
    a = dict(x=FAKE, dtype=1, rows=4, cols=128, q=FAKE, scale=FAKE)
    a.update(kw)
    assert moe.lib().moe_quantize_int8(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(q_dtype=1), UNSUPPORTED),
    (dict(q_dtype=-1), UNSUPPORTED), (dict(T=-1), ARG), (dict(H=0), ARG), (dict(H=24), ALIGN),
    (dict(H=65552), ARG), (dict(T=1 << 26), ARG), (dict(T=1 << 25, dtype=0, H=144), ARG),
    (dict(eps=-1e-6), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(x=None), ARG), (dict(weight=None), ARG), (dict(residual=None), ARG),
    (dict(total=None), ARG), (dict(scale=None), ARG), (dict(total=FAKE, y=FAKE), ARG),
    (dict(residual=None, total=None, y=None, q=None), ARG), (dict(x=ODD16), ALIGN),
    (dict(residual=ODD16), ALIGN), (dict(weight=ODD16), ALIGN), (dict(total=ODD16), ALIGN),
    (dict(y=ODD16), ALIGN), (dict(q=ODD16), ALIGN), (dict(scale=ODD4), ALIGN)])
def test_add_rms_norm_refusals(kw, status):
    a = dict(dtype=1, q_dtype=moe.MOE_I8, T=4, H=128, x=FAKE, residual=FAKE, weight=FAKE, eps=1e-6,
             total=FAKE, y=OTHER, q=FAKE, scale=FAKE)
    a.update(kw)
    assert moe.lib().moe_add_rms_norm(*a.values(), None) == status


def test_nothing_to_do():
    L = moe.lib()
    assert L.moe_quantize_int8(None, 1, 0, 128, None, None, None) == OK
    assert L.moe_add_rms_norm(1, 3, 0, 128, None, None, FAKE, 0.0, None, None, None, None, None) == OK
    assert L.moe_expert_gemm_int8(0, 4, 64, 128, None, None, None, 0, FAKE, FAKE, FAKE, FAKE, 1, None,
                                  None) == OK
    assert L.moe_expert_gemm_int8(0, 4, 64, 128, FAKE, FAKE, None, 9, FAKE, FAKE, FAKE, FAKE, 1, None,
                                  None) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), ARG), (dict(E=0), ARG), (dict(E=1025), ARG), (dict(N=8), ARG), (dict(N=24), ARG),
    (dict(K=0), ARG), (dict(K=8), ARG), (dict(K=1 << 17), ARG), (dict(N=1 << 16, K=1 << 15), ARG),
    (dict(N=1 << 21, K=16), ARG), (dict(a_rows=7), ARG), (dict(a_rows=-1), ARG),
    (dict(index=FAKE, a_rows=-1), ARG), (dict(index=FAKE, a_rows=1 << 24), ARG),
    (dict(out_dtype=2), UNSUPPORTED), (dict(out_dtype=3), UNSUPPORTED), (dict(a=None), ARG),
    (dict(sa=None), ARG), (dict(offs=None), ARG), (dict(cnts=None), ARG), (dict(w=None), ARG),
    (dict(sw=None), ARG), (dict(out=None), ARG), (dict(a=ODD16), ALIGN), (dict(w=ODD16), ALIGN),
    (dict(out=ODD16), ALIGN), (dict(sa=ODD4), ALIGN), (dict(sw=ODD16), ALIGN),
    (dict(index=ODD4), ALIGN), (dict(offs=ODD4), ALIGN), (dict(cnts=ODD4), ALIGN)])
def test_expert_gemm_int8_refusals(kw, status):
    a = dict(rows=8, E=4, N=64, K=128, a=FAKE, sa=FAKE, index=None, a_rows=8, offs=FAKE, cnts=FAKE,
             w=FAKE, sw=FAKE, out_dtype=1, out=FAKE)
    a.update(kw)
    assert moe.lib().moe_expert_gemm_int8(*a.values(), None) == status


def test_sizes_beyond_a_grid_are_refused():
    """A block of 512 threads for each tile of the streamed kernel; the tile list in 30 bits."""
    for rows, N, K in ((1 << 28, 256, 128), (1 << 24, 4096, 112), (1 << 30, 4096, 4096)):
        args = (FAKE, FAKE, None, rows, FAKE, FAKE, FAKE, FAKE, 1, FAKE, None)
        assert moe.lib().moe_expert_gemm_int8(rows, 1, N, K, *args) == ARG


def test_expert_swiglu_int8_refusals():
    L = moe.lib()

    def call(I=128, ws=1 << 24, skip=None, odd=None, **kw):
        p = [FAKE] * 10
        if skip is not None:
            p[skip] = None
        if odd is not None:
            p[odd[0]] = odd[1]
        return L.moe_expert_swiglu_int8(ctypes.byref(_shape(**kw)), I, p[0], p[1], p[2], *p[3:9],
                                        p[9], FAKE, ws, None)

    need = L.moe_expert_swiglu_int8_workspace_bytes(ctypes.byref(_shape()), 128)
    assert need == 64 * 2 * 128 * 5 + 64 * 2 * 4
    for I in (0, 8, 24, 65552):
        assert L.moe_expert_swiglu_int8_workspace_bytes(ctypes.byref(_shape()), I) == 0
        assert call(I=I) == ARG
    assert L.moe_expert_swiglu_int8_workspace_bytes(None, 128) == 0
    assert call(ws=need - 1) == WORKSPACE
    assert call(dtype=moe.MOE_F32) == UNSUPPORTED
    assert call(dtype=moe.MOE_I8) == UNSUPPORTED
    assert call(H=24) == ARG
    assert call(T=1 << 26, k=1, H=16) == ARG
    assert L.moe_expert_swiglu_int8(None, 128, *[FAKE] * 11, 1 << 24, None) == ARG
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 9):
        assert call(skip=i) == ARG, i
    assert L.moe_expert_swiglu_int8(ctypes.byref(_shape()), 128, *[FAKE] * 10, None, 1 << 24,
                                    None) == ARG
    for i, p in ((0, ODD16), (1, ODD4), (2, ODD4), (3, ODD4), (4, ODD4), (5, ODD16), (6, ODD16),
                 (7, ODD16), (8, ODD16), (9, ODD16)):
        assert call(odd=(i, p)) == ALIGN, i


def test_binding_refuses_on_the_host():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current device"):
        moe.add_rms_norm(x, w, 1e-6)
    with pytest.raises(TypeError, match="weight"):
        moe.add_rms_norm(x, w.float(), 1e-6)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        moe.add_rms_norm(x.half(), w, 1e-6)
    with pytest.raises(ValueError, match="total needs a residual"):
        moe.add_rms_norm(x, w, 1e-6, total=x)
    with pytest.raises(ValueError, match="scale needs"):
        moe.add_rms_norm(x, w, 1e-6, scale=torch.zeros(4))
    with pytest.raises(TypeError, match="int8 or float8"):
        moe.add_rms_norm(x, w, 1e-6, q_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shape"):
        moe.add_rms_norm(x, w, 1e-6, residual=x[:2])
    with pytest.raises(ValueError, match="contiguous"):
        moe.quantize_int8(torch.zeros(64, 64).t())
    with pytest.raises(TypeError):
        moe.quantize_int8(x.half())
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    o = torch.zeros(1, dtype=torch.int32)
    wq, ws = torch.zeros(1, 16, 64, dtype=torch.int8), torch.zeros(1, 16)
    with pytest.raises(ValueError, match="current device"):
        moe.expert_gemm_int8(q, s, o, o, wq, ws)
    with pytest.raises(TypeError, match="out must be"):
        moe.expert_gemm_int8(q, s, o, o, wq, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="w_scale"):
        moe.expert_gemm_int8(q, s, o, o, wq, ws[:, :8])
    with pytest.raises(TypeError, match="row_token"):
        moe.expert_gemm_int8(q, s, o, o, wq, ws, row_token=torch.zeros(3, dtype=torch.int64))
