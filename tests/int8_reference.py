"""References in 64 bits for the integer experts and the norm, and the bounds their
results are held to. No code of the library.

Half a step of a rounding, relative to the value: bf16 2^-8 (at least 2^-134, half the
smallest step), fp32 2^-24 (2^-150), e4m3 2^-4 (2^-10 of the scale); an integer half of 1.
What the kernels hold in 64 bits (sums of up to 65536 squares, root, quotient) is off by
at most 65536 * 2^-53 < 2^-36 relative, written as SLACK below."""
import torch

SLACK = 2.0 ** -36
HALF = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float32: (2.0 ** -24, 2.0 ** -150)}


def half_step(v, dtype):
    """Bound of one rounding of v to dtype (by way of fp32 for bf16)."""
    rel, least = HALF[dtype]
    extra = 2.0 ** -24 if dtype == torch.bfloat16 else 0.0
    return v.abs() * (rel + extra + SLACK) + least + (2.0 ** -150 if extra else 0)


def norm(x, weight, eps, residual=None):
    """(t as held, y) in 64 bits."""
    t = x.double()
    if residual is not None:
        t = (t + residual.double()).to(x.dtype).double()
    return t, t * weight.double() / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)


def int8_rows(v):
    """(q, scale) of the definition for finite rows v."""
    v = v.double()
    amax = v.abs().amax(-1)
    s = torch.where(amax > 0, (amax / 127).float().double().clamp(min=2.0 ** -126), 1.0)
    return torch.round(v / s.unsqueeze(-1)), s


def check_int8_rows(q, scale, v):
    """q and scale as the quantisation of rows v known to SLACK: the scale a rounding
    from amax / 127, every value within half a step of the scale that is there."""
    v, s = v.double(), scale.double()
    amax = v.abs().amax(-1)
    want = torch.where(amax > 0, (amax / 127).clamp(min=2.0 ** -126), 1.0)
    assert ((s - want).abs() <= want * (2.0 ** -24 + 2 * SLACK)).all(), "scales"
    z = v / s.unsqueeze(-1)
    # 127.0000076: the largest value of a row whose scale was rounded down
    err = (q.double() - z).abs()
    assert (err <= 0.5 + 128 * 2 * SLACK).all(), f"off by {float(err.max())} steps"
    assert int(q.abs().max() if q.numel() else 0) <= 127


def check_e4m3_rows(q, scale, v):
    """q and scale as moe_quantize's rows of v known to SLACK."""
    v, s = v.double(), scale.double()
    C = v.shape[-1]
    full = s.repeat_interleave(128, -1)[..., :C]
    pad = torch.nn.functional.pad(v, (0, s.shape[-1] * 128 - C))
    amax = pad.view(*v.shape[:-1], -1, 128).abs().amax(-1)
    low = torch.full_like(s, 2.0 ** -126)
    m, e = torch.frexp(s)
    assert (m == 0.5).all(), "powers of two"
    assert (amax <= 448 * s * (1 + 2 * SLACK)).all()
    assert ((amax > 224 * s * (1 - 2 * SLACK)) | (s == low) | ((amax == 0) & (s == 1))).all()
    err = (q.double() * full - v).abs()
    bound = torch.maximum(v.abs() * (2.0 ** -4 + 2.0 ** -20), full * 2.0 ** -10 * (1 + 2.0 ** -20))
    assert (err <= bound).all(), f"{float((err / bound.clamp(min=1e-300)).max())} of the bound"


def scaled_sums(a, a_scale, w, w_scale):
    """fp32 values of one expert's product, bit for bit: the exact sums rounded to fp32,
    times the row's scale, times the column's. a [n, K], w [N, K] int8."""
    s = a.double() @ w.double().t()  # exact: below 2^53
    return s.float() * a_scale[:, None] * w_scale[None, :]


def gemm(a, a_scale, offsets, counts, w, w_scale, row_token, out):
    """The rows of every bucket inside out, written into out (fp32 or bf16)."""
    rows = out.shape[0]
    for e, (o, n) in enumerate(zip(offsets.tolist(), counts.tolist())):
        if n <= 0 or o < 0 or o + n > rows:
            continue
        if row_token is None:
            ae, se = a[o:o + n], a_scale[o:o + n]
        else:
            t = row_token[o:o + n].long()
            ok = (t >= 0) & (t < a.shape[0])
            t = torch.where(ok, t, 0)
            ae = a[t] * ok[:, None].to(torch.int8)
            se = torch.where(ok, a_scale[t], 0.0)
        out[o:o + n] = scaled_sums(ae, se, w[e], w_scale[e]).to(out.dtype)
    return out


def swiglu(a, a_scale, wg, sg, wd, sd):
    """One expert's FFN: (out, bound) in 64 bits. g and u are three fp32 roundings off; SiLU
    has the relative condition 1 + |g| at most and 5 * 2^-24 of its own; h is one product
    more. An inner value whose quotient is that close to a border may land on either
    side: one step of the scale times its weight. The scale itself is a rounding and h's
    error off; the result three fp32 roundings and one to bf16."""
    u24 = 2.0 ** -24
    I = wd.shape[1]
    s = a.double() @ wg.double().t()
    gu = s * a_scale.double()[:, None] * sg.double()[None, :]
    g, u = gu[:, :I], gu[:, I:]
    h = g * torch.sigmoid(g) * u
    dh = h.abs() * ((1 + g.abs()) * 3 + 5 + 3 + 1) * u24 * (1 + 2.0 ** -20) + 2.0 ** -149
    q, hs = int8_rows(h)
    amax, at = h.abs().max(1)
    ds = (dh.amax(1) / 127 + hs * u24) * 1.0001  # what the scale may be off by
    z = h / hs[:, None]
    dz = dh / hs[:, None] + z.abs() * (ds / hs)[:, None]
    flip = (z - torch.floor(z) - 0.5).abs() <= dz
    w = wd.double()
    out = (q @ w.t()) * hs[:, None] * sd.double()[None, :]
    steps = (flip.double() @ w.abs().t()) * hs[:, None] * sd.double()[None, :]
    rel = (ds / hs)[:, None] + 3 * u24
    bound = steps + (out.abs() + steps) * rel * 1.0001
    bound = bound + (out.abs() + bound) * 2.0 ** -8 + 2.0 ** -133
    return out, bound
