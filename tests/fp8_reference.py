"""The 8-bit operators and the small layer from their definitions, in 64 bits on
the CPU, with bounds on what a kernel that holds its sums in fp32 may be off.

Bounds. u = 2^-24 is half an fp32 step. A dot product of n terms held in fp32 is
off by at most n * 2^-23 * sum |terms| when every addition may lose a whole step
(matrix instructions need not round to nearest inside): ``acc``. A rounding to
bf16 is off by at most 2^-8 of the value, one to e4m3 by 2^-4 of it or, below the
smallest normal value 2^-6, by half the step 2^-9.

The 8-bit matrix instruction does not add its products in full: it takes runs of
8 products, aligns them to the largest exponent E (the sum of its factors'
exponents) of the run and drops what lies below 2^(E - 13) of each, then adds the
runs in fp32 (seen on the device: 2^8 + t loses t's bits below 2^-5, t in the same
run, and nothing with t in another run). A term of exponent E is at least 2^E, so
a run of 8 is off by less than 8 * 2^-13 * max |term| <= 2^-10 * sum |terms| of the
run: 2^-10 * sum |terms| in all."""
import numpy as np
import torch

E4M3_MAX = 448.0
F32_STEP = 2.0 ** -23
RUN8 = 2.0 ** -10


def quantize(x: np.ndarray, block_rows: int):
    """x [B, R, C] float64 -> (e4m3 values as float64, scale float64), block by block."""
    B, R, C = x.shape
    q = np.zeros_like(x)
    scale = np.zeros((B, -(-R // block_rows), -(-C // 128)))
    for b in range(B):
        for i, r in enumerate(range(0, R, block_rows)):
            for j, c in enumerate(range(0, C, 128)):
                v = x[b, r:r + block_rows, c:c + 128]
                fin = np.abs(v[np.isfinite(v)])
                amax = fin.max() if fin.size else 0.0
                p = 0
                if amax > 0:
                    p = int(np.ceil(np.log2(amax / E4M3_MAX))) - 2
                    while amax > E4M3_MAX * 2.0 ** p:
                        p += 1
                    p = max(p, -126)
                scale[b, i, j] = 2.0 ** p
                q[b, r:r + block_rows, c:c + 128] = round_e4m3(np.clip(v / 2.0 ** p, -E4M3_MAX,
                                                                       E4M3_MAX))
    return q, scale


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (|v| <= 448), ties to even; NaN stays."""
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(v)
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        return np.rint(v / step) * step


def dequantize(q: torch.Tensor, scale: torch.Tensor, block_rows: int) -> torch.Tensor:
    """e4m3 tensor [..., R, C] and its block scales as float64 on the CPU."""
    q, scale = q.cpu().to(torch.float32).double(), scale.cpu().double()
    s = scale.repeat_interleave(block_rows, -2)[..., :q.shape[-2], :]
    return q * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def product(a, w, counts, offsets, out=None):
    """(exact product, accumulation bound) of grouped rows, float64 [rows, N].
    a [rows, K], w [E, N, K] float64; rows outside the buckets are zero."""
    rows, K = a.shape
    N = w.shape[1]
    ref = torch.zeros(rows, N, dtype=torch.float64)
    acc = torch.zeros(rows, N, dtype=torch.float64)
    for e, (n, o) in enumerate(zip(counts.tolist(), offsets.tolist())):
        if n:
            ref[o:o + n] = a[o:o + n] @ w[e].t()
            # K products and additions, then one multiply-add a block with a
            # rounded product of scales
            acc[o:o + n] = ((K + 3 * (K // 128 + 1)) * F32_STEP + RUN8) * (a[o:o + n].abs()
                                                                           @ w[e].abs().t())
    return ref, acc


def swiglu(g, u, dg, du):
    """(h, bound) of silu(g) u from g, u known to dg, du: |silu'| <= 1.1, silu and
    the product rounded to a few fp32 steps."""
    s = g * torch.sigmoid(g)
    h = s * u
    ds = 1.1 * dg + 2.0 ** -21 * s.abs()
    return h, ds * (u.abs() + du) + s.abs() * du + 2.0 ** -22 * h.abs()


def route(logits, k):
    """(idx, gate) of float64 logits: descending, the lower id on ties."""
    order = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(logits, order, 1)
    w = np.exp(top - top[:, :1])
    return order, w / w.sum(1, keepdims=True)


def layer(logits, x, k, wg, wd):
    """(idx, gate, y, bound of |y_kernel - y|): float64 logits [T, E], x [T, H],
    wg [E, 2I, H], wd [E, H, I]. h is rounded to bf16, y too."""
    idx, gate = route(logits.numpy(), k)
    T, H = x.shape
    I = wd.shape[2]
    y = torch.zeros(T, H, dtype=torch.float64)
    bound = torch.zeros(T, H, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for i in range(k):
            e, w = int(idx[t, i]), float(gate[t, i])
            gu = wg[e] @ x[t]
            d = (H + 3 * (H // 64 + 1)) * F32_STEP * (wg[e].abs() @ x[t].abs())
            h, dh = swiglu(gu[:I], gu[I:], d[:I], d[I:])
            dh = dh + 2.0 ** -8 * (h.abs() + dh)  # rounded to bf16
            y[t] += w * (wd[e] @ h)
            m = wd[e].abs() @ (h.abs() + dh)
            bound[t] += w * (wd[e].abs() @ dh)
            mag[t] += w * m
    # fp32 sums over I and over the picks, the gate weight's own rounding
    bound += (I + 3 * (I // 64 + 1) + 4 * k + 16) * F32_STEP * mag
    return idx, gate, y, bound + 2.0 ** -8 * (y.abs() + bound)
