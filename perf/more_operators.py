"""The integer expert path and the norm that feeds it, as cases to measure.

Each case names one operator, its sizes and its routing. ``run`` computes it in
plain torch operations, or, where ``own`` is true, with the calls of
``combine_moe_route_03_amd``; ``exact`` computes it from the definition in 64
bits. The sizes are those of this repository's workloads (decode_hot, zipf,
dirichlet_waves, local_layer) and ranges around them.

Operators:
  norm      t = x + residual, y = t / sqrt(mean(t^2) + eps) * weight, and y in 8 bits: int8
            with a scale a row, or e4m3 with a power-of-two scale a 128 columns
  quantize  x -> (int8 values, scale of each row: amax / 127)
  gemm      each expert's int8 rows times its int8 weights, with a scale for each row and for
            each column of the result; the rows lie in expert order or are picked by index
  swiglu    the SwiGLU expert FFN on int8 rows and weights, its inner rows in int8 as well
"""
import math

import torch

own = False

_DEV = "cuda:0"
_EPS = 1e-6


def listed():
    return [
        # Decoding one sequence: the norm before the router, rows out in int8. Latency.
        {"name": "norm-one", "op": "norm", "T": 1, "H": 4096, "q": "int8", "want_y": True,
         "residual": True, "dtype": "bf16"},
        # A decode batch whose experts take e4m3 blocks.
        {"name": "norm-decode-e4m3", "op": "norm", "T": 128, "H": 4096, "q": "e4m3",
         "want_y": True, "residual": True, "dtype": "bf16"},
        # The largest workload's tokens (dirichlet_waves).
        {"name": "norm-prefill", "op": "norm", "T": 16384, "H": 7168, "q": "int8", "want_y": True,
         "residual": True, "dtype": "bf16"},
        # A ragged batch of fp32 rows, as an FFN's inner rows are.
        {"name": "quantize-rows", "op": "quantize", "rows": 4093, "cols": 1408, "dtype": "f32"},
        # The local layer's gate/up weights, one scale a channel, when a model is loaded.
        {"name": "quantize-weights", "op": "quantize", "rows": 16 * 2816, "cols": 4096,
         "dtype": "bf16"},
        # A dense projection of five tokens: the weights are all there is to read.
        {"name": "gemm-dense-few", "op": "gemm", "T": 5, "E": 1, "k": 1, "N": 4096, "K": 7168,
         "routing": "iid", "gather": False, "out": "bf16"},
        # Gate/up product of a decode batch, its tokens picked by index.
        {"name": "gemm-decode", "op": "gemm", "T": 128, "E": 128, "k": 8, "N": 2816, "K": 4096,
         "routing": "hot", "gather": True, "out": "bf16"},
        # Down product of a ragged prefill batch: odd row counts, partial tiles.
        {"name": "gemm-ragged", "op": "gemm", "T": 4093, "E": 64, "k": 6, "N": 2048, "K": 1408,
         "routing": "zipf", "gather": False, "out": "bf16"},
        # A dense layer's product over a long prefill.
        {"name": "gemm-dense", "op": "gemm", "T": 8192, "E": 1, "k": 1, "N": 4096, "K": 7168,
         "routing": "iid", "gather": False, "out": "bf16"},
        # One token through its experts.
        {"name": "swiglu-one", "op": "swiglu", "T": 1, "E": 128, "k": 8, "H": 4096, "I": 1408,
         "routing": "iid", "gather": True},
        # The decode batch through its experts, most picks on a few hot ones.
        {"name": "swiglu-decode", "op": "swiglu", "T": 128, "E": 128, "k": 8, "H": 4096,
         "I": 1408, "routing": "hot", "gather": True},
        # The local layer.
        {"name": "swiglu-local", "op": "swiglu", "T": 8192, "E": 16, "k": 2, "H": 4096,
         "I": 1408, "routing": "zipf", "gather": True},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, min(hi, int(round(v / step)) * step))

    op = rng.choice(["norm", "quantize", "gemm", "swiglu"])
    if op == "norm":
        return {"op": op, "T": log(1, 8192), "H": log(128, 7168, 16),
                "q": rng.choice(["int8", "e4m3", ""]), "want_y": True,
                "residual": rng.random() < 0.75, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "quantize":
        return {"op": op, "rows": log(1, 20000), "cols": log(64, 7168, 16),
                "dtype": rng.choice(["bf16", "f32"])}
    routing = rng.choice(["iid", "zipf", "hot"])
    E, k = log(16, 128), rng.randint(1, 8)
    if op == "gemm":
        if rng.random() < 0.4:
            E, k, routing = 1, 1, "iid"
        N, K = log(128, 4096, 16), log(128, 7168, 16)
        T = log(1, min(8192, 240_000_000_000 // (k * N * K)))  # at most the dense layer's work
        return {"op": op, "T": T, "E": E, "k": k, "N": N, "K": K, "routing": routing,
                "gather": E > 1 and rng.random() < 0.5, "out": rng.choice(["bf16", "bf16", "f32"])}
    H, I = log(512, 4096, 16), log(128, 1408, 16)
    T = log(1, min(8192, 90_000_000_000 // (k * H * I)))  # at most the local layer's
    return {"op": op, "T": T, "E": E, "k": k, "H": H, "I": I, "routing": routing,
            "gather": rng.random() < 0.7}


# ------------------------------------------------------------------ inputs

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _router_logits(T, E, k, routing, g):
    """Router logits [T, E]: independent, with a Zipf bias over a random order
    of the experts, or with four fifths of the picks on eight hot experts."""
    noise = torch.randn(T, E, generator=g, device=_DEV)
    if routing == "zipf":
        rank = torch.randperm(E, generator=g, device=_DEV) + 1
        return noise - 0.5 * rank.float().log()
    if routing == "hot":
        order = torch.randperm(E, generator=g, device=_DEV)
        on_hot = (torch.rand(T, k, generator=g, device=_DEV) < 0.8).sum(1, keepdim=True)
        place = torch.rand(T, E, generator=g, device=_DEV)
        hot, cold = order[:8], order[8:]
        boost = torch.zeros_like(noise)
        boost[:, hot] = (place[:, hot].argsort(1).argsort(1) < on_hot).float()
        boost[:, cold] = (place[:, cold].argsort(1).argsort(1) < k - on_hot).float()
        return noise + 8.0 * boost
    return noise


def _buckets(logits, k):
    """Picks in expert order (token order inside an expert): counts and offsets of
    the experts and the token of every row."""
    E = logits.shape[1]
    picks = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k].reshape(-1)
    order = torch.sort(picks, stable=True)[1]
    counts = torch.bincount(picks, minlength=E)
    offsets = torch.cumsum(counts, 0) - counts
    return counts.int(), offsets.int(), (order // k).int()


def _int8_rows(x):
    """Rows as a calibrated program holds them: scale amax / 127."""
    s = x.float().abs().amax(-1) / 127
    return (x.float() / s.unsqueeze(-1)).round().clamp_(-127, 127).to(torch.int8), s


def _int8_weights(E, N, K, g):
    """Weights of a checkpoint in 8-bit integers, one scale for each channel."""
    q = torch.empty(E, N, K, device=_DEV, dtype=torch.int8)
    scale = torch.empty(E, N, device=_DEV)
    step = max(1, (1 << 28) // (N * K))  # experts at a time: bounds the 32-bit copies
    for e in range(0, E, step):
        w = torch.randn(min(step, E - e), N, K, generator=g, device=_DEV).mul_(0.02)
        q[e:e + step], scale[e:e + step] = _int8_rows(w)
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)

    def hidden(rows, cols):
        # rows of different size, as hidden states have
        x = torch.randn(rows, cols, generator=g, device=_DEV)
        return x * torch.exp(torch.randn(rows, 1, generator=g, device=_DEV))

    if op == "norm":
        T, H, dt = case["T"], case["H"], _DTYPES[case["dtype"]]
        s["x"] = hidden(T, H).to(dt)
        s["r"] = hidden(T, H).to(dt) if case["residual"] else None
        s["w"] = (1 + 0.1 * torch.randn(H, generator=g, device=_DEV)).to(dt)
        s["total"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y"] = torch.empty_like(s["x"]) if case["want_y"] else None
        s["q8"], s["scale"] = None, None
        if case["q"]:
            qt = torch.int8 if case["q"] == "int8" else torch.float8_e4m3fn
            s["q8"] = torch.empty(T, H, device=_DEV, dtype=qt)
            s["scale"] = torch.empty((T,) if case["q"] == "int8" else (T, -(-H // 128)),
                                     device=_DEV)
        return s
    if op == "quantize":
        s["x"] = hidden(case["rows"], case["cols"]).to(_DTYPES[case["dtype"]])
        s["q8"] = torch.empty(s["x"].shape, device=_DEV, dtype=torch.int8)
        s["scale"] = torch.empty(case["rows"], device=_DEV)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    logits = _router_logits(T, E, k, case["routing"], g)
    s["counts"], s["offsets"], token = _buckets(logits, k)
    s["most"] = int(s["counts"].max())  # the longest expert's rows
    K = case["K"] if op == "gemm" else case["H"]
    s["a"], s["a_scale"] = _int8_rows(hidden(T if case["gather"] else T * k, K))
    s["row_token"] = token if case["gather"] else None
    if op == "gemm":
        s["w"], s["w_scale"] = _int8_weights(E, case["N"], K, g)
        s["y"] = torch.empty(T * k, case["N"], device=_DEV, dtype=_DTYPES[case["out"]])
    else:
        s["w_gate_up"], s["s_gate_up"] = _int8_weights(E, 2 * case["I"], K, g)
        s["w_down"], s["s_down"] = _int8_weights(E, K, case["I"], g)
        s["y"] = torch.empty(T * k, K, device=_DEV, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------- plain forms

def _quantize_int8(x):
    """Rows of x (any floating type) to int8: scale amax / 127 as fp32 (1 for a row
    of zeros), values x / scale to the nearest, ties to even. In 64 bits, so that a
    value next to a border between two integers lands on its own side."""
    x = x.double()
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, (amax / 127).float().clamp(min=2.0 ** -126), 1.0)
    q = torch.round(x / scale.double().unsqueeze(-1)).clamp(-127, 127)
    return q.to(torch.int8), scale


def _quantize_e4m3(x):
    """Groups of 128 columns to e4m3 with the scale 2^p, p the smallest >= -126
    with amax <= 448 * 2^p (p = 0 for a group of zeros)."""
    R, C = x.shape
    cb = -(-C // 128)
    v = torch.nn.functional.pad(x, (0, cb * 128 - C)).view(R, cb, 128)
    amax = v.abs().amax(2)
    m, e = torch.frexp(amax)
    p = torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(min=-126), 0).int()
    inverse = ((127 - p) << 23).view(torch.float32).double()
    scale = ((127 + p) << 23).view(torch.float32)
    q = (v * inverse.unsqueeze(2)).clamp(-448, 448).reshape(R, cb * 128)[:, :C]
    return q.float().to(torch.float8_e4m3fn), scale


def _grouped(a, counts, offsets, most, w):
    """Rows of expert e times w[e]^T, over the experts' rows laid side by side."""
    slot = torch.arange(most, device=a.device)
    row = (offsets[:, None] + slot[None, :]).long()
    live = slot[None, :] < counts[:, None]
    out = torch.bmm(a[torch.where(live, row, 0)], w.transpose(1, 2))
    return out[live]  # expert order is row order


def _by_expert(values, counts):
    """values [E, N] for each row: its expert's."""
    return values.repeat_interleave(counts.long(), 0)


def _product(s, a, a_scale, w, w_scale):
    # Whole products in 32 bits: off by at most 2^-24 of what is summed a step.
    if a.shape[0] < w.shape[0]:  # fewer rows than experts: each row by its own expert
        e = torch.arange(w.shape[0], device=_DEV).repeat_interleave(s["counts"].long())
        p = torch.bmm(w[e].float(), a.float().unsqueeze(2)).squeeze(2)
        return p * a_scale.unsqueeze(1) * w_scale[e]
    p = _grouped(a.float(), s["counts"], s["offsets"], s["most"], w.float())
    return p * a_scale.unsqueeze(1) * _by_expert(w_scale, s["counts"])


def _plain(s):
    op = s["op"]
    if op == "norm":
        total = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
        # 64 bits: the 8-bit values next to a border
        v = total.double()
        y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS) * s["w"].double()
        q, scale = None, None
        if s["q"]:
            q, scale = _quantize_int8(y) if s["q"] == "int8" else _quantize_e4m3(y)
        return (None if s["r"] is None else total, y.to(s["x"].dtype) if s["want_y"] else None,
                q, scale)
    if op == "quantize":
        return _quantize_int8(s["x"])
    a, a_scale = s["a"], s["a_scale"]
    if s["row_token"] is not None:
        at = s["row_token"].long()
        a, a_scale = a[at], a_scale[at]
    if op == "gemm":
        return _product(s, a, a_scale, s["w"], s["w_scale"]).to(s["y"].dtype)
    gu = _product(s, a, a_scale, s["w_gate_up"], s["s_gate_up"])
    g, u = gu[:, :s["I"]], gu[:, s["I"]:]
    hq, hs = _quantize_int8(g / (1 + torch.exp(-g)) * u)
    return _product(s, hq, hs, s["w_down"], s["s_down"]).to(torch.bfloat16)


# --------------------------------------------------- the framework's calls

def _own(s):
    import combine_moe_route_03_amd as moe

    op = s["op"]
    if op == "norm":
        return moe.add_rms_norm(s["x"], s["w"], _EPS, residual=s["r"], total=s["total"],
                                y=s["y"], want_y=s["want_y"], q=s["q8"], scale=s["scale"])
    if op == "quantize":
        return moe.quantize_int8(s["x"], q=s["q8"], scale=s["scale"])
    if op == "gemm":
        return moe.expert_gemm_int8(s["a"], s["a_scale"], s["offsets"], s["counts"], s["w"],
                                    s["w_scale"], row_token=s["row_token"], out=s["y"])
    shape = moe.Shape(s["T"], s["H"], s["E"], s["k"], 1, 1, torch.bfloat16)
    if "workspace" not in s:  # kept by the caller from step to step
        need = moe.expert_swiglu_int8_workspace_bytes(shape, s["I"])
        s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device=_DEV)
    return moe.expert_swiglu_int8(s["a"], s["a_scale"], s["offsets"], s["counts"], shape,
                                  s["w_gate_up"], s["s_gate_up"], s["w_down"], s["s_down"],
                                  row_token=s["row_token"], expert_out=s["y"],
                                  workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# -------------------------------------------------------------------- work

def _live_experts(case):
    """Experts with a pick, on average (as if the picks of a Zipf bias were even)."""
    T, E, k = case["T"], case["E"], case["k"]
    if case["routing"] == "hot":
        return 8 + (E - 8) * (1 - (1 - min(1.0, 0.2 * k / (E - 8))) ** T)
    return E * (1 - (1 - k / E) ** T)


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        b = 2 if case["dtype"] == "bf16" else 4
        per = b * (1 + 2 * case["residual"] + case["want_y"]) + (1 if case["q"] else 0)
        scales = T * {"int8": 1, "e4m3": -(-H // 128), "": 0}[case["q"]]
        return {"bytes": T * H * per + H * b + 4 * scales, "flops": 8 * T * H}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (3 if case["dtype"] == "bf16" else 5) + 4 * case["rows"],
                "flops": 3 * n}
    T, E, k = case["T"], case["E"], case["k"]
    rows = T * k
    live = _live_experts(case)
    read = (T if case["gather"] else rows)
    index = 4 * rows if case["gather"] else 0
    if op == "gemm":
        N, K = case["N"], case["K"]
        b = 2 if case["out"] == "bf16" else 4
        return {"bytes": read * (K + 4) + index + rows * N * b + live * N * (K + 4),
                "flops": 2 * rows * N * K}
    H, I = case["H"], case["I"]
    return {"bytes": read * (H + 4) + index + rows * 2 * H + live * (3 * H * I + 8 * I + 4 * H),
            "flops": 6 * rows * H * I}


# ------------------------------------------------------------------- exact

def _exact_int8(x):
    """Each row by its own scale: the nearest 32-bit number to amax / 127."""
    q, scale = torch.empty_like(x), torch.ones(x.shape[0], dtype=torch.float64, device=x.device)
    for r in range(0, x.shape[0], 4096):
        rows = x[r:r + 4096]
        top = torch.maximum(rows.amax(1), -rows.amin(1))
        s = (top / 127).to(torch.float32).to(torch.float64)
        s = torch.where(top == 0, 1.0, torch.maximum(s, torch.full_like(s, 2.0 ** -126)))
        scale[r:r + 4096] = s
        q[r:r + 4096] = (rows / s[:, None]).round()
    return q, scale


def _power_of_two(e):
    """2^e in 64 bits, from its bit pattern (pow and ldexp may be an ulp off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(x):
    """The blocks from the definition: the scale from the binary exponent of
    amax / 448, each value to the nearest multiple of its binade's step."""
    q = torch.empty_like(x)
    scale = torch.empty(x.shape[0], -(-x.shape[1] // 128), dtype=torch.float64, device=x.device)
    for j in range(scale.shape[1]):
        cols = x[:, 128 * j:128 * (j + 1)]
        f, e = torch.frexp(cols.abs().amax(1) / 448.0)  # f in [0.5, 1)
        s = _power_of_two(torch.where(f > 0.5, e, e - 1))
        s = torch.where(f > 0, s.clamp(min=2.0 ** -126), 1.0)
        v = cols / s[:, None]
        _, e = torch.frexp(v)
        step = _power_of_two((e - 1).clamp(min=-6) - 3)
        q[:, 128 * j:128 * (j + 1)] = torch.round(v / step) * step
        scale[:, j] = s
    return q, scale


def _exact_product(a, a_scale, w, w_scale):
    """One expert: the integers' sums (exact in 64 bits), then both scales."""
    return (a @ w.double().t()) * (a_scale.double()[:, None] * w_scale.double()[None, :])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        t = s["x"].double()
        if s["r"] is not None:
            # what is normalised is the sum as it is held
            t = (t + s["r"].double()).to(s["x"].dtype).double()
        size = torch.linalg.vector_norm(t, dim=1, keepdim=True)
        y = s["w"].double() * (t / torch.sqrt(size * size / case["H"] + _EPS))
        q, scale = None, None
        if case["q"]:
            q, scale = _exact_int8(y) if case["q"] == "int8" else _exact_e4m3(y)
        return t if s["r"] is not None else None, y if case["want_y"] else None, q, scale
    if op == "quantize":
        return _exact_int8(s["x"].double())
    out = torch.empty(s["y"].shape, dtype=torch.float64, device=_DEV)
    for e, (n, o) in enumerate(zip(s["counts"].tolist(), s["offsets"].tolist())):
        if n == 0:
            continue
        at = torch.arange(o, o + n, device=_DEV) if s["row_token"] is None else (
            s["row_token"][o:o + n].long())
        a, sa = s["a"][at].double(), s["a_scale"][at]
        if op == "gemm":
            out[o:o + n] = _exact_product(a, sa, s["w"][e], s["w_scale"][e])
        else:
            gu = _exact_product(a, sa, s["w_gate_up"][e], s["s_gate_up"][e])
            g, u = gu[:, :case["I"]], gu[:, case["I"]:]
            hq, hs = _exact_int8(g * torch.sigmoid(g) * u)
            out[o:o + n] = _exact_product(hq, hs, s["w_down"][e], s["s_down"][e])
    return out
