"""The 8-bit experts on the GPU against their definitions in 64 bits: block
quantisation and the quantising dispatch bit for bit, the grouped product and
the SwiGLU FFN within bounds derived from their roundings (fp8_reference.py),
and the operators in a row as a model runs them."""
import numpy as np
import pytest
import torch

import combine_moe_route_03_amd as moe
import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(*shape, seed=0, scale=1.0):
    return torch.randn(*shape, generator=gen(seed)) * scale


def fp8_weights(E, N, K, seed, std=0.05):
    """e4m3 weights with scales that are no powers of two."""
    w = torch.randn(E, N, K, generator=gen(seed)) * std
    nb, kb = -(-N // 128), -(-K // 128)
    s = torch.rand(E, nb, kb, generator=gen(seed + 1)) * 0.003 + 0.0007
    wide = s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return (w / wide).clamp(-448, 448).to(F8), s


def buckets(counts, gap=0):
    c = torch.tensor(counts, dtype=torch.int32)
    o = torch.zeros_like(c)
    at = 0
    for i, n in enumerate(counts):
        o[i] = at
        at += n + (gap if n else 0)
    return c, o, at


# ------------------------------------------------------------------ quantise

def special_rows(rows, cols, seed):
    """Normal rows of many sizes with zeros, infinities, NaN, denormals, ties and
    block maxima on both sides of 448 * 2^p."""
    x = torch.randn(rows, cols, generator=gen(seed)).numpy()
    x *= np.exp2(np.arange(rows) % 40 - 20)[:, None].astype(np.float32)
    for r in range(rows):
        kind = r % 10
        if kind == 1:
            x[r] = 0
        elif kind == 2:
            x[r, :: 7] = np.inf
        elif kind == 3:
            x[r, 1:: 5] = np.nan
            x[r, 2:: 5] = -np.inf
        elif kind == 4:
            x[r] = np.sign(x[r]) * 1e-39
        elif kind == 5:
            x[r] = np.nan
        elif kind == 6:  # halfway between e4m3 values, and the subnormal ones
            x[r] = (np.arange(cols) % 256 - 128) * 2.0 ** -10 * 1.0
            x[r, 0] = 448 * 2.0 ** (r % 8)
        elif kind == 7:
            x[r, 0] = 449.0
        elif kind == 8:
            x[r, 3] = 3.0e38
    return torch.from_numpy(x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("batch,rows,cols", [
    (1, 1, 16), (1, 1, 128), (1, 3, 144), (2, 130, 256), (3, 127, 1424), (1, 128, 128),
    (5, 1, 4096), (1, 257, 272)])
def test_quantize(batch, rows, cols, block_rows, dtype):
    print(f"[quantize] {batch}x{rows}x{cols} block_rows={block_rows} {dtype}", flush=True)
    x = special_rows(batch * rows, cols, 3).view(batch, rows, cols).to(dtype)
    q, s = moe.quantize(x.to(DEV), block_rows=block_rows)
    with np.errstate(all="ignore"):
        rq, rs = ref.quantize(x.double().numpy(), block_rows)
    assert np.array_equal(s.cpu().double().numpy(), rs)
    got = q.cpu().float().double().numpy()
    assert np.array_equal(got, rq, equal_nan=True)


def test_quantize_every_bf16():
    """Every bf16 bit pattern in a block whose scale is 1: e4m3 rounding itself."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[bits.float().abs() <= 448]
    x = x[: x.numel() // 112 * 112].view(-1, 112)
    x = torch.cat([torch.full((x.shape[0], 16), 448.0, dtype=torch.bfloat16), x], 1)
    q, s = moe.quantize(x.contiguous().to(DEV))
    assert bool((s == 1).all())
    assert np.array_equal(q.cpu().float().double().numpy(), ref.round_e4m3(x.double().numpy()))


def test_quantize_empty():
    q, s = moe.quantize(torch.empty(0, 128, device=DEV))
    assert q.shape == (0, 128) and s.shape == (0, 1)


# ------------------------------------------------------------------ dispatch

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,E,k", [(1, 128, 8, 2), (7, 144, 16, 8), (33, 2048, 64, 6),
                                     (5, 16, 64, 32), (200, 7168, 32, 3)])
def test_dispatch_copy_fp8(T, H, E, k, dtype):
    print(f"[dispatch fp8] T={T} H={H} E={E} k={k} {dtype}", flush=True)
    x = special_rows(T, H, 5).to(dtype)
    logits = randn(T, E, seed=6)
    shape = moe.Shape(T, H, E, k, 1, 1, dtype)
    idx, _ = moe.route(logits.to(DEV), k)
    idx[0, 0] = -1  # a dropped pick: no row
    d = moe.alloc_dispatch(shape, DEV)
    moe.dispatch_index(idx, shape, d)
    q = torch.full((T * k, H), 7.0, device=DEV).to(F8)
    s = torch.full((T * k, -(-H // 128)), -5.0, device=DEV)
    moe.dispatch_copy_fp8(x.to(DEV), d["pos"], shape, send_q=q, send_scale=s)
    with np.errstate(all="ignore"):
        rq, rs = ref.quantize(x.double().numpy()[None], 1)
    eq, es = np.full((T * k, H), 7.0), np.full((T * k, rs.shape[2]), -5.0)
    pos = d["pos"].cpu().numpy()
    for t in range(T):
        for i in range(k):
            if pos[t, i] >= 0:
                eq[pos[t, i]], es[pos[t, i]] = rq[0, t], rs[0, t]
    assert np.array_equal(s.cpu().double().numpy(), es)
    assert np.array_equal(q.cpu().float().double().numpy(), eq, equal_nan=True)


# ------------------------------------------------------------------ product

GEMM = [
    # counts, gap, N, K
    ([1], 0, 16, 128), ([1], 0, 256, 256), ([300], 0, 272, 384), ([0, 1, 0, 2, 255, 256, 257], 0, 128, 128),
    ([3, 0, 17, 64, 65], 5, 144, 640), ([16] * 9, 0, 2816, 1408), ([513, 1], 3, 1024, 512),
    ([5] * 70, 0, 48, 256), ([40, 33, 0, 12], 0, 512, 8448), ([700], 0, 640, 128),
    # several tiles a compute unit: two, three and five K steps, row tiles of few
    # rows between full ones, columns past the last tile, K steps beyond 64
    ([3000], 0, 8192, 256), ([2900], 0, 7952, 384), ([700, 0, 513, 1, 1, 600], 2, 4112, 640),
    ([30, 0, 29, 257, 1] * 9, 0, 2064, 384), ([90, 40], 0, 272, 8576), ([33] * 300, 1, 256, 256),
]


@pytest.mark.parametrize("counts,gap,N,K", GEMM)
def test_expert_gemm_fp8(counts, gap, N, K):
    print(f"[gemm fp8] counts={counts[:8]} gap={gap} N={N} K={K}", flush=True)
    E = len(counts)
    c, o, rows = buckets(counts, gap)
    rows += 4  # rows behind the last bucket
    a, sa = moe.quantize((randn(rows, K, seed=1) * torch.exp(randn(rows, 1, seed=2))).to(DEV))
    sa = sa * (torch.rand(sa.shape, generator=gen(3)) + 0.5).to(DEV)  # any scales
    w, sw = fp8_weights(E, N, K, 4)
    out = torch.full((rows, N), -77.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_gemm_fp8(a, sa, o.to(DEV), c.to(DEV), w.to(DEV), sw.to(DEV), out=out)
    r, acc = ref.product(ref.dequantize(a, sa, 1), ref.dequantize(w, sw, 128), c, o)
    got = out.cpu().double()
    live = torch.zeros(rows, dtype=torch.bool)
    for n, b in zip(c.tolist(), o.tolist()):
        live[b:b + n] = True
    assert bool((got[~live] == -77.0).all())
    err = (got - r).abs() - (acc + 2.0 ** -8 * (r.abs() + acc))
    assert float(err[live].max()) <= 0, f"{float(err[live].max())} over the bound"
    # all in all no more than the rounding to bf16 can take from every value: what
    # the instruction drops has either sign and nearly cancels over the runs
    assert float((got - r)[live].norm()) <= 2.0 ** -8 * float(r[live].norm())


def test_expert_gemm_fp8_buckets_outside_the_rows_are_ignored():
    c = torch.tensor([4, 9, 3, 5], dtype=torch.int32, device=DEV)
    o = torch.tensor([0, 100, -2, 14], dtype=torch.int32, device=DEV)  # only the first lies inside
    a, sa = moe.quantize(randn(16, 128, seed=1).to(DEV))
    w, sw = fp8_weights(4, 64, 128, 2)
    out = torch.full((16, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_gemm_fp8(a, sa, o, c, w.to(DEV), sw.to(DEV), out=out)
    assert bool((out[4:] == 3.0).all()) and not bool((out[:4] == 3.0).all())


def test_expert_gemm_fp8_bad_buckets_among_many_rows():
    """The same with many rows an expert: counts and offsets that leave the rows."""
    c = torch.tensor([130, 100, 7, 5000], dtype=torch.int32, device=DEV)
    o = torch.tensor([10, 250, -2, 0], dtype=torch.int32, device=DEV)  # only the first lies inside
    a, sa = moe.quantize(randn(300, 256, seed=1).to(DEV))
    w, sw = [t.to(DEV) for t in fp8_weights(4, 64, 256, 2)]
    out = torch.full((300, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_gemm_fp8(a, sa, o, c, w, sw, out=out)
    assert bool((out[:10] == 3.0).all()) and bool((out[140:] == 3.0).all())
    o[1:], c[1:] = 0, 0
    only = torch.full_like(out, 3.0)
    moe.expert_gemm_fp8(a, sa, o, c, w, sw, out=only)
    assert torch.equal(out, only) and not bool((out[10:140] == 3.0).all())


@pytest.mark.parametrize("rows", [20, 600])
def test_expert_gemm_fp8_counts_beyond_the_rows_end(rows):
    """Every expert claims all rows (no routing does): the list of tiles stays as long as
    that of buckets that do not overlap, and what is written is an expert's product."""
    E = 5
    a, sa = moe.quantize(randn(rows, 256, seed=1).to(DEV))
    w, sw = [t.to(DEV).expand(E, -1, -1).contiguous() for t in fp8_weights(1, 64, 256, 2)]
    o, c = (torch.full((E,), v, dtype=torch.int32, device=DEV) for v in (0, rows))
    out = moe.expert_gemm_fp8(a, sa, o, c, w, sw)
    one = moe.expert_gemm_fp8(a, sa, o[:1], c[:1], w[:1], sw[:1])
    assert torch.equal(out, one)


def test_expert_gemm_fp8_nan_stays_in_its_row():
    a, sa = moe.quantize(randn(40, 256, seed=1).to(DEV))
    clean = moe.expert_gemm_fp8(a, sa, *[t.to(DEV) for t in buckets([40])[1::-1]],
                                *[t.to(DEV) for t in fp8_weights(1, 128, 256, 2)])
    a.view(torch.uint8)[17, 33] = 0x7F  # NaN
    out = moe.expert_gemm_fp8(a, sa, *[t.to(DEV) for t in buckets([40])[1::-1]],
                              *[t.to(DEV) for t in fp8_weights(1, 128, 256, 2)])
    keep = torch.arange(40, device=DEV) != 17
    assert bool(out[17].isnan().all()) and torch.equal(out[keep], clean[keep])


def test_without_rows():
    """No tokens: every entry returns empty outputs and touches nothing."""
    shape = moe.Shape(0, 256, 4, 2, 1, 1, torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    q, s = moe.dispatch_copy_fp8(torch.empty(0, 256, dtype=torch.bfloat16, device=DEV),
                                 torch.empty(0, 2, dtype=torch.int32, device=DEV), shape)
    (wg, sg), (wd, sd) = [[t.to(DEV) for t in fp8_weights(4, *nk, 2)] for nk in ((256, 256), (256, 128))]
    assert moe.expert_gemm_fp8(q, s, i, i, wg, sg).shape == (0, 256)
    assert moe.expert_swiglu_fp8(q, s, i, i, shape, wg, sg, wd, sd).shape == (0, 256)
    # rows, but no expert has any
    a, sa = moe.quantize(torch.ones(300, 256, device=DEV))
    out = torch.full((300, 256), 4.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_gemm_fp8(a, sa, i, i, wg, sg, out=out)
    moe.expert_gemm_fp8(a[:8], sa[:8], i, i, wg, sg, out=out[:8])
    assert bool((out == 4.0).all())


def e4m3_bytes(*shape, seed):
    """Random e4m3 values made on the device (no NaN)."""
    g = torch.Generator(DEV).manual_seed(seed)
    b = torch.randint(0, 240, shape, dtype=torch.uint8, device=DEV, generator=g)
    b.bitwise_xor_((b & 1) << 7)  # signs
    return b.bitwise_and_(0xF7).view(F8)


def test_rows_and_weights_past_32_bits():
    """More than 2^32 bytes of rows, of weights and of send rows: the last ones as alone."""
    K, N, n = 2048, 32, 300
    rows = (1 << 32) // K + 5000
    a = e4m3_bytes(rows, K, seed=1)
    sa = torch.rand(rows, K // 128, device=DEV) + 0.5
    w, sw = [t.to(DEV) for t in fp8_weights(1, N, K, 3)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    out = moe.expert_gemm_fp8(a, sa, i32(0), i32(rows), w, sw)
    alone = moe.expert_gemm_fp8(a[-n:], sa[-n:], i32(0), i32(n), w, sw)
    assert torch.equal(out[-n:], alone)
    del a, sa, out
    E, N = 520, 4096
    w = e4m3_bytes(E, N, K, seed=2)
    sw = torch.rand(E, N // 128, K // 128, device=DEV) + 0.5
    for n in (7, 40):  # streamed, and (all the rows in one bucket of many) tiled
        rows = n if n == 7 else 28 * E + 256
        a, sa = moe.quantize(randn(rows, K, seed=4).to(DEV))
        o, c = torch.zeros(E, dtype=torch.int32, device=DEV), torch.zeros(E, dtype=torch.int32, device=DEV)
        c[-1] = n
        out = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
        moe.expert_gemm_fp8(a, sa, o, c, w, sw, out=out)
        a1 = a[:rows if n == 7 else 300].contiguous()
        alone = torch.zeros(len(a1), N, dtype=torch.bfloat16, device=DEV)
        moe.expert_gemm_fp8(a1, sa[:len(a1)].contiguous(), o[-1:], c[-1:], w[-1:].contiguous(),
                            sw[-1:].contiguous(), out=alone)
        assert torch.equal(out[:n], alone[:n]) and not bool((out[:n] == 0).all())
        assert not bool(out[n:].any())
    del w, sw
    shape = moe.Shape(70000, 8192, 8, 8, 1, 1, torch.bfloat16)
    x = torch.randn(shape.T, shape.H, dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(shape.T * 8, dtype=torch.int32, device=DEV).view(-1, 8).flip(0).contiguous()
    q, s = moe.dispatch_copy_fp8(x, pos, shape)
    xq, xs = moe.quantize(x)
    for t in (0, 1, shape.T // 2, shape.T - 1):
        for r in pos[t].tolist():
            assert torch.equal(q[r].view(torch.uint8), xq[t].view(torch.uint8)) and torch.equal(s[r], xs[t])


# ------------------------------------------------------------------ FFN

@pytest.mark.parametrize("counts,H,I", [
    ([1], 128, 128), ([0, 3, 260, 0, 1], 256, 384), ([17, 64, 1], 1024, 128),
    ([6] * 20, 384, 1408), ([300, 280], 512, 256), ([60, 0, 300, 1, 20] * 5, 256, 1408),
    ([2100], 384, 2176), ([30, 270] * 3, 128, 640)])
def test_expert_swiglu_fp8(counts, H, I):
    print(f"[swiglu fp8] counts={counts[:6]} H={H} I={I}", flush=True)
    E, rows = len(counts), sum(counts)
    c, o, _ = buckets(counts)
    shape = moe.Shape(rows, H, E, 1, 1, 1, torch.bfloat16)
    a, sa = moe.quantize(randn(rows, H, seed=1).to(DEV))
    wg, sg = fp8_weights(E, 2 * I, H, 2)
    wd, sd = fp8_weights(E, H, I, 4)
    ws = torch.zeros(moe.expert_swiglu_fp8_workspace_bytes(shape, I), dtype=torch.uint8, device=DEV)
    out = moe.expert_swiglu_fp8(a, sa, o.to(DEV), c.to(DEV), shape, wg.to(DEV), sg.to(DEV),
                                wd.to(DEV), sd.to(DEV), workspace=ws)
    # the 8-bit intermediate: h to within its own error and one e4m3 rounding
    gu, acc = ref.product(ref.dequantize(a, sa, 1), ref.dequantize(wg, sg, 128), c, o)
    h, dh = ref.swiglu(gu[:, :I], gu[:, I:], acc[:, :I], acc[:, I:])
    hq = ws[:rows * I].view(F8).view(rows, I)
    at = max(256, -(-rows * I // 256) * 256)
    hs = ws[at:at + rows * (I // 128) * 4].view(torch.float32).view(rows, I // 128)
    scale = hs.cpu().double()
    amax = h.abs().view(rows, I // 128, 128).amax(2)
    assert bool(torch.isfinite(scale).all()) and bool((torch.frexp(scale)[0] == 0.5).all())
    dmax = dh.view(rows, I // 128, 128).amax(2)  # the kernel's maximum is this near
    assert bool((amax - dmax <= 448 * scale).all()) and bool((amax + dmax > 224 * scale).all())
    wide = scale.repeat_interleave(128, 1)
    dq = dh + 2.0 ** -4 * (h.abs() + dh) + 2.0 ** -10 * wide
    assert float(((ref.dequantize(hq, hs, 1) - h).abs() - dq).max()) <= 0
    # the down product of what the workspace holds
    r, acc = ref.product(ref.dequantize(hq, hs, 1), ref.dequantize(wd, sd, 128), c, o)
    err = (out.cpu().double() - r).abs() - (acc + 2.0 ** -8 * (r.abs() + acc))
    assert float(err.max()) <= 0, f"{float(err.max())} over the bound"
    assert float((out.cpu().double() - r).norm()) <= 2.0 ** -8 * float(r.norm())


# ------------------------------------------------------------ a run of them

def test_route_dispatch_ffn_combine_in_8_bits():
    """Weights quantised in blocks, rows quantised by the dispatch, the FFN and the
    framework's combine: the result is the bf16 layer's to within what 8 bits
    lose. Every value passes three roundings to e4m3 (x and w of each product, h
    between), each off by 2^-4 of it at most, so g and u are off by (2^-3 + 2^-8)
    of the sums of magnitudes, and so on; the bound is the one of those sums."""
    T, H, E, k, I = 37, 256, 8, 3, 256
    shape = moe.Shape(T, H, E, k, 2, 2, torch.bfloat16)
    x = randn(T, H, seed=1).to(torch.bfloat16)
    wg = randn(E, 2 * I, H, seed=2, scale=0.06).to(torch.bfloat16)
    wd = randn(E, H, I, seed=3, scale=0.06).to(torch.bfloat16)
    idx, gate = moe.route(randn(T, E, seed=4).to(DEV), k)
    d = moe.alloc_dispatch(shape, DEV)
    moe.dispatch_index(idx, shape, d)
    sq, ss = moe.dispatch_copy_fp8(x.to(DEV), d["pos"], shape)
    qg, sg = moe.quantize(wg.to(DEV), block_rows=128)
    qd, sd = moe.quantize(wd.to(DEV), block_rows=128)
    eo = moe.expert_swiglu_fp8(sq, ss, d["expert_offsets"], d["expert_counts"], shape, qg, sg, qd, sd)
    y = moe.combine(eo, gate, d["pos"], shape).cpu().double()
    xs, wgs, wds = x.double(), wg.double(), wd.double()
    off8 = 2.0 ** -4
    for t in range(T):
        want, bound = torch.zeros(H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
        for i in range(k):
            e, w = int(idx[t, i]), float(gate[t, i])
            gu, mag = wgs[e] @ xs[t], wgs[e].abs() @ xs[t].abs()
            # subnormal steps: half of 2^-9 of a scale that is at most 2^-7 of the block maximum
            small = 2.0 ** -10 * 2.0 ** -7
            dx, dw = float(xs[t].abs().max()) * small, float(wgs[e].abs().max()) * small
            dgu = (2 * off8 + off8 ** 2 + 2 * ref.RUN8) * mag + dx * wgs[e].abs().sum(1) \
                + dw * xs[t].abs().sum() * (1 + off8)
            h, dh = ref.swiglu(gu[:I], gu[I:], dgu[:I], dgu[I:])
            dh = dh + off8 * (h.abs() + dh) + small * float((h.abs() + dh).max())
            dwd = off8 * wds[e].abs() + small * float(wds[e].abs().max())
            want += w * (wds[e] @ h)
            bound += w * (wds[e].abs() @ dh + dwd @ (h.abs() + dh))
        # the second product's runs (2^-10 of sums of which bound holds 2^-4), and the bf16
        # roundings of expert_out and y
        bound = bound * (1 + 2.0 ** -5) + 2.0 ** -6 * want.abs()
        assert float(((y[t] - want).abs() - bound).max()) <= 0


def test_streams_and_graphs():
    """The FFN on a side stream, and two captured graphs with a workspace each,
    replayed in turn with eager work between, give the eager bits."""
    counts, H, I = [30, 0, 5, 130], 256, 256
    E, rows = len(counts), sum(counts)
    c, o, _ = buckets(counts)
    c, o = c.to(DEV), o.to(DEV)
    shape = moe.Shape(rows, H, E, 1, 1, 1, torch.bfloat16)
    wg, sg = [t.to(DEV) for t in fp8_weights(E, 2 * I, H, 2)]
    wd, sd = [t.to(DEV) for t in fp8_weights(E, H, I, 4)]
    xs = [randn(rows, H, seed=10 + i).to(DEV) for i in range(2)]
    nbytes = moe.expert_swiglu_fp8_workspace_bytes(shape, I)

    def bufs():
        return dict(q=torch.empty(rows, H, dtype=F8, device=DEV), s=torch.empty(rows, H // 128, device=DEV),
                    ws=torch.empty(nbytes, dtype=torch.uint8, device=DEV),
                    out=torch.empty(rows, H, dtype=torch.bfloat16, device=DEV))

    def step(x, b):
        moe.quantize(x, q=b["q"], scale=b["s"])
        moe.expert_swiglu_fp8(b["q"], b["s"], o, c, shape, wg, sg, wd, sd, expert_out=b["out"],
                              workspace=b["ws"])

    want = []
    for x in xs:
        b = bufs()
        step(x, b)
        torch.cuda.synchronize()
        want.append(b["out"].clone())
    side = torch.cuda.Stream()
    b = bufs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xs[0], b)
    torch.cuda.synchronize()
    assert torch.equal(b["out"], want[0])
    graphs = []
    for x in xs:
        b = bufs()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            step(x, b)
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                step(x, b)
        graphs.append((g, b))
    eager = bufs()
    for rep in range(3):
        for (g, b), w in zip(graphs, want):
            b["out"].fill_(9.0)
            step(xs[rep % 2], eager)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(b["out"], w), rep
