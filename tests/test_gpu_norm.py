"""The norm with the residual's addition and its 8-bit rows, and the integer quantisation
of rows, against their definitions in 64 bits (int8_reference.py has the bounds)."""
import pytest
import torch

import combine_moe_route_03_amd as moe
import int8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn

# every lane layout: part of a wave, a wave, blocks of one to sixteen vectors a lane
WIDTHS = [16, 48, 128, 144, 256, 400, 512, 528, 1408, 4096, 4112, 7168, 8208, 16384, 20480, 65536]


def hidden(T, H, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV) * torch.exp(
        2 * torch.randn(T, 1, generator=g, device=DEV))
    return x.to(dtype)


def check_norm(x, w, eps, r, q_dtype, got):
    total, y, q, scale = got
    t, want = ref.norm(x, w, eps, r)
    if r is not None:
        assert torch.equal(total.double(), t)
    else:
        assert total is None
    if y is not None:
        assert ((y.double() - want).abs() <= ref.half_step(want, x.dtype)).all()
    if q_dtype == torch.int8:
        ref.check_int8_rows(q, scale, want)
    elif q_dtype == E4M3:
        ref.check_e4m3_rows(q, scale, want)


@pytest.mark.parametrize("q_dtype", [None, torch.int8, E4M3])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, dtype, q_dtype):
    for T, add in ((1, True), (5, False), (17, True)):
        print(f"[norm] T={T} H={H} {dtype} q={q_dtype} residual={add}", flush=True)
        x = hidden(T, H, dtype, 1)
        w = (1 + 0.3 * torch.randn(H, device=DEV)).to(dtype)
        r = hidden(T, H, dtype, 2) if add else None
        got = moe.add_rms_norm(x, w, 1e-5, residual=r, q_dtype=q_dtype)
        check_norm(x, w, 1e-5, r, q_dtype, got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [48, 144, 272, 528, 784, 1040, 1408, 2064, 2832, 4080, 4112, 8192])
def test_rows_of_a_wave(H, dtype):
    """From 1024 rows on a wave takes a row, up to eight vectors a lane."""
    for T, add, q_dtype in ((1024, True, torch.int8), (1027, False, E4M3), (1030, True, None)):
        x, r = hidden(T, H, dtype, 21), hidden(T, H, dtype, 22) if add else None
        w = (1 + 0.3 * torch.randn(H, device=DEV)).to(dtype)
        check_norm(x, w, 1e-5, r, q_dtype, moe.add_rms_norm(x, w, 1e-5, residual=r, q_dtype=q_dtype))
    q, scale = moe.quantize_int8(x)
    want_q, want_s = ref.int8_rows(x)
    assert torch.equal(scale.double(), want_s) and torch.equal(q.double(), want_q)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_rows(dtype):
    """More rows than a wave of blocks, past the size up to which results are cached."""
    T, H = (24001, 4096) if dtype == BF16 else (9001, 4096)
    x, r = hidden(T, H, dtype, 3), hidden(T, H, dtype, 4)
    w = (1 + 0.1 * torch.randn(H, device=DEV)).to(dtype)
    got = moe.add_rms_norm(x, w, 1e-6, residual=r, q_dtype=torch.int8)
    for a in range(0, T, 8192):  # bounds the 64-bit copies
        check_norm(x[a:a + 8192], w, 1e-6, r[a:a + 8192], torch.int8,
                   tuple(v[a:a + 8192] for v in got))


def test_only_what_is_asked_for():
    x, r = hidden(9, 1024, BF16, 5), hidden(9, 1024, BF16, 6)
    w = torch.ones(1024, device=DEV, dtype=BF16)
    full = moe.add_rms_norm(x, w, 1e-6, residual=r, q_dtype=torch.int8)
    some = moe.add_rms_norm(x, w, 1e-6, residual=r, q_dtype=torch.int8, want_y=False)
    assert some[1] is None and torch.equal(some[0], full[0])
    assert torch.equal(some[2], full[2]) and torch.equal(some[3], full[3])
    plain = moe.add_rms_norm(full[0], w, 1e-6)
    assert plain[0] is None and plain[2] is None and torch.equal(plain[1], full[1])
    shaped = moe.add_rms_norm(x.view(3, 3, 1024), w, 1e-6, residual=r.view(3, 3, 1024), q_dtype=E4M3)
    assert shaped[1].shape == (3, 3, 1024) and shaped[3].shape == (3, 3, 8)
    assert torch.equal(shaped[1].view(9, 1024), full[1])
    empty = moe.add_rms_norm(x[:0], w, 1e-6, residual=r[:0], q_dtype=torch.int8)
    assert empty[1].shape == (0, 1024) and empty[3].shape == (0,)


@pytest.mark.parametrize("H", [128, 512, 4096, 16384])
@pytest.mark.parametrize("total_in,y_in", [("r", None), ("x", None), ("r", "x"), ("x", "r")])
def test_in_place(H, total_in, y_in):
    x, r = hidden(7, H, BF16, 7), hidden(7, H, BF16, 8)
    w = (1 + 0.1 * torch.randn(H, device=DEV)).to(BF16)
    want = moe.add_rms_norm(x, w, 1e-6, residual=r, q_dtype=torch.int8)
    b = {"x": x.clone(), "r": r.clone()}
    got = moe.add_rms_norm(b["x"], w, 1e-6, residual=b["r"], q_dtype=torch.int8, total=b[total_in],
                           y=b[y_in] if y_in else None)
    for g, v in zip(got, want):
        assert torch.equal(g, v)
    assert got[0] is b[total_in]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [128, 512, 4096])
def test_values_at_the_ends(H, dtype):
    """Rows of zeros, of the largest values (whose squares pass fp32), of the smallest,
    one value alone; a row does not touch its neighbours."""
    x = hidden(9, H, dtype, 9)
    big = torch.finfo(dtype).max
    x[1] = 0
    x[2] = big
    x[2, 1::2] = -big
    x[3] = x[3] * 1e-38
    x[4] = 0
    x[4, H - 1] = 3.0
    x[5] = 2.0 ** -133
    w = (1 + 0.1 * torch.randn(H, device=DEV)).to(dtype)
    w[3] = 0
    for eps in (1e-6, 1e-20):
        for q_dtype in (torch.int8, E4M3):
            check_norm(x, w, eps, None, q_dtype, moe.add_rms_norm(x, w, eps, q_dtype=q_dtype))
    # without eps a row of zeros has no norm
    total, y, q, scale = moe.add_rms_norm(x, w, 0.0, q_dtype=torch.int8)
    assert y[1].isnan().all() and scale[1].isnan() and (q[1] == 0).all()
    keep = [0, 2, 3, 4, 5, 6, 7, 8]
    check_norm(x[keep], w, 0.0, None, torch.int8, (None, y[keep], q[keep], scale[keep]))


@pytest.mark.parametrize("T,H", [(6, 128), (6, 512), (6, 4096), (1050, 512), (1050, 2048), (1050, 8192)])
def test_infinities_and_nan(T, H):
    inf, nan = float("inf"), float("nan")
    x = hidden(T, H, BF16, 10)
    w = (1 + 0.1 * torch.randn(H, device=DEV)).to(BF16)
    clean = moe.add_rms_norm(x, w, 1e-6, q_dtype=torch.int8)
    clean8 = moe.add_rms_norm(x, w, 1e-6, q_dtype=E4M3)
    bad = x.clone()
    bad[1, 5] = inf
    bad[3, H - 1] = nan
    total, y, q, scale = moe.add_rms_norm(bad, w, 1e-6, q_dtype=torch.int8)
    assert y[1, 5].isnan() and (y[1, :5] == 0).all() and (y[1, 6:] == 0).all()
    assert y[3].isnan().all()
    for i in (1, 3):
        assert scale[i].isnan() and (q[i] == 0).all()
    y8, q8, s8 = moe.add_rms_norm(bad, w, 1e-6, q_dtype=E4M3)[1:]
    assert q8[1, 5].float().isnan() and (q8[1, :5].float() == 0).all() and s8[1, 0] == 1
    assert q8[3].float().isnan().all()
    for i in (0, 2, 4, 5, T - 1):
        assert torch.equal(y[i], clean[1][i]) and torch.equal(q[i], clean[2][i])
        assert torch.equal(q8[i].view(torch.uint8), clean8[2][i].view(torch.uint8))
    # an infinite weight: infinities saturate, the others keep the scale of the finite ones
    wi = w.clone()
    wi[7] = inf
    w0 = w.clone()
    w0[7] = 0
    y, q, scale = moe.add_rms_norm(x, wi, 1e-6, q_dtype=torch.int8)[1:]
    q0, s0 = moe.add_rms_norm(x, w0, 1e-6, q_dtype=torch.int8)[2:]
    live = x[:, 7] != 0
    assert (y[live, 7].abs() == inf).all()
    assert torch.equal(scale[live], s0[live])
    assert torch.equal(q[live, 7].float(), 127 * x[live, 7].float().sign())
    q0[:, 7] = q[:, 7]
    assert torch.equal(q[live], q0[live])


@pytest.mark.parametrize("T", [1, 1030])
def test_int8_next_to_a_border(T):
    """Quotients 2^-37 to 2^-44 off the middle of two integers land on their own side: t w is
    the product of two 24-bit integers next to (2 n + 1) 2^44, the row's norm a power of two."""
    g = torch.Generator().manual_seed(17)
    a = torch.randint(1 << 23, 1 << 24, (1 << 21,), generator=g)
    t, w, want = [127.0], [1.0], [127]
    for n in range(1, 8):
        m = (2 * n + 1) << 44
        b = (m + a // 2) // a
        d = a * b - m
        for below in (True, False):
            ok = (d < 0 if below else d > 0) & (d.abs() < 256) & (b < 1 << 24)
            i = int(ok.nonzero()[0])
            for sign in (1, -1):
                t.append(sign * float(a[i]) * 2.0 ** -23)
                w.append(float(b[i]) * 2.0 ** -22)
                want.append(sign * (n if below else n + 1))
    t, w = torch.tensor(t + [0.0] * 3, dtype=F32), torch.tensor(w + [1.0] * 3, dtype=F32)
    assert t.numel() == 32
    eps = 1024.0 - float((t.double() ** 2).mean())
    x = t.to(DEV).repeat(T, 1)
    _, _, q, scale = moe.add_rms_norm(x, w.to(DEV), eps, q_dtype=torch.int8)
    assert (scale == 2.0 ** -5).all()
    assert torch.equal(q.cpu(), torch.tensor(want + [0] * 3, dtype=torch.int8).repeat(T, 1))


# ------------------------------------------------------------------ quantize_int8

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_quantize_widths(cols, dtype):
    for rows in (1, 6, 35):
        print(f"[quantize int8] {rows}x{cols} {dtype}", flush=True)
        x = hidden(rows, cols, dtype, 11)
        q, scale = moe.quantize_int8(x)
        want_q, want_s = ref.int8_rows(x)
        assert torch.equal(scale.double(), want_s)
        assert torch.equal(q.double(), want_q)


def test_quantize_borders():
    """Quotients half way between two integers, and next to there."""
    g = torch.Generator().manual_seed(12)
    for scale in (1.0, 0.75, 2.0 ** -126, 2.0 ** 100, 5 / 8):
        half = (torch.arange(-127, 127) + 0.5) * scale
        x = torch.zeros(3, 512)
        x[:, :254] = half
        x[1, :254] = torch.nextafter(half, torch.full_like(half, float("inf")))
        x[2, :254] = torch.nextafter(half, torch.full_like(half, -float("inf")))
        x[:, 300] = 127 * scale
        x[:, 301:] = scale * 127 * (2 * torch.rand(3, 211, generator=g) - 1)
        q, s = moe.quantize_int8(x.to(DEV))
        want_q, want_s = ref.int8_rows(x)
        assert torch.equal(s.cpu().double(), want_s) and (want_s == scale).all()
        assert torch.equal(q.cpu().double(), want_q), scale


def test_quantize_random_borders():
    """Any scale: values one step of fp32 around every half quotient."""
    g = torch.Generator().manual_seed(13)
    amax = torch.exp(8 * torch.randn(64, 1, generator=g))
    s = (amax.double() / 127).float()
    half = ((torch.arange(-126, 126) + 0.5).double() * s.double()).float()
    x = torch.cat([half, torch.nextafter(half, half * 2), torch.nextafter(half, half * 0),
                   amax, torch.zeros(64, 11)], 1)
    assert x.shape[1] == 768
    q, scale = moe.quantize_int8(x.to(DEV))
    want_q, want_s = ref.int8_rows(x)
    assert torch.equal(scale.cpu().double(), want_s) and torch.equal(q.cpu().double(), want_q)


def test_quantize_values_at_the_ends():
    inf, nan = float("inf"), float("nan")
    for cols in (64, 512, 4096):
        x = hidden(8, cols, F32, 14)
        x[1] = 0
        x[2] = 0
        x[2, 3] = 2.0 ** -149
        x[3, 0], x[3, 1] = inf, -inf
        x[4, 9] = nan
        x[5] = torch.finfo(F32).max
        x[6] = inf
        q, s = moe.quantize_int8(x)
        assert s[1] == 1 and (q[1] == 0).all()
        assert s[2] == 2.0 ** -126 and (q[2] == 0).all()
        finite = x[3].clone()
        finite[:2] = 0
        want_q, want_s = ref.int8_rows(finite.unsqueeze(0))
        assert s[3].double() == want_s[0] and torch.equal(q[3, 2:].double(), want_q[0, 2:])
        assert q[3, 0] == 127 and q[3, 1] == -127
        assert s[4].isnan() and (q[4] == 0).all()
        assert (q[5] == 127).all() and s[5].isfinite()
        assert s[6] == 1 and (q[6] == 127).all()  # no finite value
        for i in (0, 7):
            want_q, want_s = ref.int8_rows(x[i:i + 1])
            assert torch.equal(q[i].double(), want_q[0]) and s[i].double() == want_s[0]


def test_quantize_weights_and_large():
    w = hidden(6 * 96, 1408, BF16, 15).view(6, 96, 1408)
    q, s = moe.quantize_int8(w)
    assert q.shape == w.shape and s.shape == (6, 96)
    want_q, want_s = ref.int8_rows(w)
    assert torch.equal(q.double(), want_q) and torch.equal(s.double(), want_s)
    x = hidden(40001, 4096, BF16, 16)  # past the size up to which results are cached
    q, s = moe.quantize_int8(x)
    for a in range(0, 40001, 8192):
        want_q, want_s = ref.int8_rows(x[a:a + 8192])
        assert torch.equal(q[a:a + 8192].double(), want_q)
        assert torch.equal(s[a:a + 8192].double(), want_s)
