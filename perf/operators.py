"""The 8-bit expert path and the few-token MoE layer, as cases to measure.

Each case names one operator, its sizes and its routing. ``run`` computes it in
plain torch operations in 32 bits, or, where ``own`` is true, with the calls of
``combine_moe_route_03_amd``; ``exact`` computes it from the definition in 64
bits. The sizes are those of this repository's workloads (decode_hot, zipf,
dirichlet_waves, local_layer) and ranges around them.

Operators:
  quantize   x -> (e4m3 values, power-of-two scale of each 1 x 128 or 128 x 128 block)
  dispatch   the permute copy of token rows, quantised on the way
  gemm       each expert's rows times its weights, both e4m3 with block scales
  swiglu     the SwiGLU expert FFN on e4m3 rows and weights
  layer      routing, experts and combine of a few tokens, from logits to y
"""
import math

import torch

own = False

_DEV = "cuda:0"
_FP8_MAX = 448.0  # largest finite e4m3 value


def listed():
    return [
        # A decode batch's hidden states before an 8-bit product: latency.
        {"name": "quantize-rows-decode", "op": "quantize", "batch": 1, "rows": 128, "cols": 4096,
         "block_rows": 1, "dtype": "bf16"},
        # The local layer's gate/up weights, converted once when a model is loaded.
        {"name": "quantize-blocks-weights", "op": "quantize", "batch": 16, "rows": 2816,
         "cols": 4096, "block_rows": 128, "dtype": "bf16"},
        # Prefill rows of the zipf workload, packed in 8 bits for the exchange.
        {"name": "dispatch-zipf", "op": "dispatch", "T": 4096, "H": 2048, "E": 64, "k": 6,
         "routing": "zipf", "dtype": "bf16"},
        # The largest workload's exchange: 131072 rows of 7168.
        {"name": "dispatch-waves", "op": "dispatch", "T": 16384, "H": 7168, "E": 256, "k": 8,
         "routing": "zipf", "dtype": "bf16"},
        # Gate/up product of a decode batch: few rows an expert, weights bound.
        {"name": "gemm-decode", "op": "gemm", "T": 128, "E": 128, "k": 8, "N": 2816, "K": 4096,
         "routing": "hot"},
        # Down product of a ragged prefill batch: odd row counts, partial tiles.
        {"name": "gemm-ragged", "op": "gemm", "T": 4093, "E": 64, "k": 6, "N": 2048, "K": 1408,
         "routing": "zipf"},
        # One expert: a dense layer's product.
        {"name": "gemm-dense", "op": "gemm", "T": 8192, "E": 1, "k": 1, "N": 4096, "K": 7168,
         "routing": "iid"},
        # The FFN of a decode batch.
        {"name": "swiglu-decode", "op": "swiglu", "T": 128, "E": 128, "k": 8, "H": 4096,
         "I": 1408, "routing": "hot"},
        # The FFN of the local layer.
        {"name": "swiglu-local", "op": "swiglu", "T": 8192, "E": 16, "k": 2, "H": 4096,
         "I": 1408, "routing": "zipf"},
        # One token through a layer: the smallest decode step.
        {"name": "layer-one", "op": "layer", "T": 1, "H": 4096, "E": 128, "k": 8, "I": 1408,
         "weights": "bf16", "routing": "iid"},
        # A small batch with 8-bit weights.
        {"name": "layer-few-fp8", "op": "layer", "T": 17, "H": 2048, "E": 64, "k": 6, "I": 1408,
         "weights": "fp8", "routing": "iid"},
        # The whole decode batch, most picks on a few hot experts.
        {"name": "layer-decode", "op": "layer", "T": 128, "H": 4096, "E": 128, "k": 8, "I": 1408,
         "weights": "bf16", "routing": "hot"},
    ]


def draw(rng):
    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, min(hi, int(round(v / step)) * step))

    op = rng.choice(["quantize", "dispatch", "gemm", "swiglu", "layer"])
    routing = rng.choice(["iid", "zipf", "hot"])
    if op == "quantize":
        block_rows = rng.choice([1, 128])
        return {"op": op, "batch": log(1, 16), "rows": log(1, 2816), "cols": log(16, 4096, 16),
                "block_rows": block_rows, "dtype": rng.choice(["bf16", "f32"])}
    if op == "dispatch":
        E = log(16, 256)
        return {"op": op, "T": log(1, 8192), "H": log(128, 7168, 128), "E": E,
                "k": rng.randint(1, 8), "routing": routing, "dtype": rng.choice(["bf16", "f32"])}
    E = log(16, 128)
    k = rng.randint(1, 8)
    if op == "gemm":
        if rng.random() < 0.25:
            E, k, routing = 1, 1, "iid"
        T = log(1, 4096)
        N, K = log(128, 4096, 16), log(128, 4096, 128)
        return {"op": op, "T": T, "E": E, "k": k, "N": N, "K": K, "routing": routing}
    H, I = log(512, 4096, 128), log(128, 1408, 128)
    if op == "swiglu":
        return {"op": op, "T": log(1, 4096), "E": E, "k": min(k, 2 + 8 * (E < 64)), "H": H,
                "I": I, "routing": routing}
    return {"op": op, "T": log(1, 128), "H": H, "E": E, "k": k, "I": I,
            "weights": rng.choice(["bf16", "fp8"]), "routing": routing}


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
    """Picks in expert order (token order inside an expert): counts, offsets and
    the row of every pick."""
    E = logits.shape[1]
    picks = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k].reshape(-1)
    order = torch.sort(picks, stable=True)[1]
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=_DEV)
    counts = torch.bincount(picks, minlength=E)
    offsets = torch.cumsum(counts, 0) - counts
    return counts.int(), offsets.int(), pos.view(-1, k).int()


def _weights(E, N, K, g):
    return torch.randn(E, N, K, generator=g, device=_DEV, dtype=torch.bfloat16).mul_(0.02)


def _weights_fp8(E, N, K, g):
    """Block-scaled weights as a checkpoint brings them: scale amax / 448."""
    nb, kb = -(-N // 128), -(-K // 128)
    q = torch.empty(E, N, K, device=_DEV, dtype=torch.float8_e4m3fn)
    scale = torch.empty(E, nb, kb, device=_DEV)
    step = max(1, (1 << 28) // (N * K))  # experts at a time: bounds the 32-bit copies
    for e in range(0, E, step):
        w = _weights(min(step, E - e), N, K, g).float()
        w = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nb * 128 - N))
        w = w.view(-1, nb, 128, kb, 128)
        s = w.abs().amax((2, 4)) / _FP8_MAX
        w = (w / s[:, :, None, :, None]).clamp_(-_FP8_MAX, _FP8_MAX)
        q[e:e + step] = w.view(-1, nb * 128, kb * 128)[:, :N, :K].to(torch.float8_e4m3fn)
        scale[e:e + step] = s
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "quantize":
        dt = _DTYPES[case["dtype"]]
        lead = (case["batch"], case["rows"])
        x = torch.randn(*lead, case["cols"], generator=g, device=_DEV)
        # rows of different size, as hidden states have
        x *= torch.exp(torch.randn(*lead, 1, generator=g, device=_DEV))
        s["x"] = x.to(dt)
        s["q"] = torch.empty(x.shape, device=_DEV, dtype=torch.float8_e4m3fn)
        s["scale"] = torch.empty(case["batch"], -(-case["rows"] // case["block_rows"]),
                                 -(-case["cols"] // 128), device=_DEV)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    logits = _router_logits(T, E, k, case["routing"], g)
    if op == "layer":
        H, I = case["H"], case["I"]
        s["logits"] = logits
        s["x"] = torch.randn(T, H, generator=g, device=_DEV).to(torch.bfloat16)
        if case["weights"] == "fp8":
            s["w_gate_up"], s["s_gate_up"] = _weights_fp8(E, 2 * I, H, g)
            s["w_down"], s["s_down"] = _weights_fp8(E, H, I, g)
        else:
            s["w_gate_up"], s["s_gate_up"] = _weights(E, 2 * I, H, g), None
            s["w_down"], s["s_down"] = _weights(E, H, I, g), None
        s["y"] = torch.empty(T, H, device=_DEV, dtype=torch.bfloat16)
        return s
    counts, offsets, pos = _buckets(logits, k)
    s["counts"], s["offsets"], s["pos"] = counts, offsets, pos
    rows = T * k
    s["most"] = int(counts.max())  # the longest expert's rows
    if op == "dispatch":
        x = torch.randn(T, case["H"], generator=g, device=_DEV)
        s["x"] = (x * torch.exp(torch.randn(T, 1, generator=g, device=_DEV))).to(
            _DTYPES[case["dtype"]])
        s["send_q"] = torch.empty(rows, case["H"], device=_DEV, dtype=torch.float8_e4m3fn)
        s["send_scale"] = torch.empty(rows, -(-case["H"] // 128), device=_DEV)
        return s
    K = case["K"] if op == "gemm" else case["H"]
    x = torch.randn(rows, K, generator=g, device=_DEV)
    s["a"], s["a_scale"] = _quantize(x.to(torch.bfloat16).unsqueeze(0), 1)
    s["a"], s["a_scale"] = s["a"][0], s["a_scale"][0]
    if op == "gemm":
        s["w"], s["w_scale"] = _weights_fp8(E, case["N"], K, g)
        s["out"] = torch.empty(rows, case["N"], device=_DEV, dtype=torch.bfloat16)
    else:
        I = case["I"]
        s["w_gate_up"], s["s_gate_up"] = _weights_fp8(E, 2 * I, K, g)
        s["w_down"], s["s_down"] = _weights_fp8(E, K, I, g)
        s["out"] = torch.empty(rows, K, device=_DEV, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------- plain forms

def _quantize(x, block_rows):
    """x [B, R, C] -> e4m3 values and the power-of-two scale 2^p of each block:
    the smallest p >= -126 with amax <= 448 * 2^p (0 for a block of zeros)."""
    x = x.float()
    B, R, C = x.shape
    rb, cb = -(-R // block_rows), -(-C // 128)
    v = torch.nn.functional.pad(x, (0, cb * 128 - C, 0, rb * block_rows - R))
    v = v.view(B, rb, block_rows, cb, 128)
    amax = torch.where(v.isfinite(), v.abs(), 0.0).amax((2, 4))
    m, e = torch.frexp(amax)
    p = torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(min=-126), 0).int()
    inverse = ((127 - p) << 23).view(torch.float32)[:, :, None, :, None]
    scale = ((127 + p) << 23).view(torch.float32)
    q = (v * inverse).clamp(-_FP8_MAX, _FP8_MAX).reshape(B, rb * block_rows, cb * 128)
    return q[:, :R, :C].to(torch.float8_e4m3fn), scale


def _dequantize(q, scale, block_rows):
    s = scale.repeat_interleave(block_rows, -2)[..., :q.shape[-2], :]
    s = s.repeat_interleave(128, -1)[..., :q.shape[-1]]
    return q.float() * s


def _grouped(a, counts, offsets, most, w):
    """Rows of expert e times w[e]^T, over the experts' rows laid side by side."""
    slot = torch.arange(most, device=a.device)
    row = (offsets[:, None] + slot[None, :]).long()
    live = slot[None, :] < counts[:, None]
    out = torch.bmm(a[torch.where(live, row, 0)], w.transpose(1, 2))
    return out[live]  # expert order is row order


def _silu(g):
    return g / (1 + torch.exp(-g))


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _quantize(s["x"], s["block_rows"])
    if op == "dispatch":
        q, scale = _quantize(s["x"].unsqueeze(0), 1)
        token = torch.empty(s["pos"].numel(), dtype=torch.long, device=_DEV)
        token[s["pos"].view(-1).long()] = (
            torch.arange(token.numel(), device=_DEV) // s["k"])
        return q[0].view(torch.uint8)[token].view(torch.float8_e4m3fn), scale[0][token]
    if op == "gemm":
        a = _dequantize(s["a"], s["a_scale"], 1)
        w = _dequantize(s["w"], s["w_scale"], 128)
        return _grouped(a, s["counts"], s["offsets"], s["most"], w).to(torch.bfloat16)
    if op == "swiglu":
        a = _dequantize(s["a"], s["a_scale"], 1)
        w = _dequantize(s["w_gate_up"], s["s_gate_up"], 128)
        gu = _grouped(a, s["counts"], s["offsets"], s["most"], w)
        del w
        h = _silu(gu[:, :s["I"]]) * gu[:, s["I"]:]
        hq, hs = _quantize(h.unsqueeze(0), 1)
        h = _dequantize(hq[0], hs[0], 1)
        w = _dequantize(s["w_down"], s["s_down"], 128)
        return _grouped(h, s["counts"], s["offsets"], s["most"], w).to(torch.bfloat16)
    logits, x, k, I = s["logits"], s["x"].float(), s["k"], s["I"]
    T, E = logits.shape
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = idx[:, :k]
    top = top[:, :k].double()
    gate = torch.exp(top - top[:, :1])
    gate = (gate / gate.sum(1, keepdim=True)).float()
    wg, wd, sg, sd = s["w_gate_up"], s["w_down"], s["s_gate_up"], s["s_down"]
    if T * k < E:  # each pick's own expert
        pick = idx.reshape(-1)
        xe = x.repeat_interleave(k, 0).unsqueeze(1)
        if sg is not None:
            wg, wd = wg.view(torch.uint8)[pick].view(wg.dtype), wd.view(torch.uint8)[pick].view(
                wd.dtype)
            wg, wd = _dequantize(wg, sg[pick], 128), _dequantize(wd, sd[pick], 128)
        else:
            wg, wd = wg[pick].float(), wd[pick].float()
        gu = torch.bmm(xe, wg.transpose(1, 2))
        h = _silu(gu[..., :I]) * gu[..., I:]
        o = torch.bmm(h, wd.transpose(1, 2)).view(T, k, -1)
        y = (gate.unsqueeze(-1) * o).sum(1)
    else:  # every expert on every token, weighted by its gate (0 where not picked)
        dense = torch.zeros(T, E, device=_DEV).scatter_(1, idx, gate)
        wg = wg.float() if sg is None else _dequantize(wg, sg, 128)
        gu = torch.bmm(x.expand(E, T, -1), wg.transpose(1, 2))
        del wg
        h = _silu(gu[..., :I]) * gu[..., I:] * dense.t().unsqueeze(-1)
        wd = wd.float() if sd is None else _dequantize(wd, sd, 128)
        y = torch.bmm(h, wd.transpose(1, 2)).sum(0)
    return y.to(torch.bfloat16), idx.int(), gate


# --------------------------------------------------- the framework's calls

def _workspace(s, nbytes):
    if "workspace" not in s:  # kept by the caller from step to step
        s["workspace"] = torch.empty(max(nbytes(), 1), dtype=torch.uint8, device=_DEV)
    return s["workspace"]


def _own(s):
    import combine_moe_route_03_amd as moe

    op = s["op"]
    if op == "quantize":
        return moe.quantize(s["x"], block_rows=s["block_rows"], q=s["q"], scale=s["scale"])
    if op == "dispatch":
        shape = moe.Shape(s["T"], s["H"], s["E"], s["k"], 1, 1, s["x"].dtype)
        return moe.dispatch_copy_fp8(s["x"], s["pos"], shape, send_q=s["send_q"],
                                     send_scale=s["send_scale"])
    if op == "gemm":
        return moe.expert_gemm_fp8(s["a"], s["a_scale"], s["offsets"], s["counts"], s["w"],
                                   s["w_scale"], out=s["out"])
    if op == "swiglu":
        shape = moe.Shape(s["T"], s["H"], s["E"], s["k"], 1, 1, torch.bfloat16)
        ws = _workspace(s, lambda: moe.expert_swiglu_fp8_workspace_bytes(shape, s["I"]))
        return moe.expert_swiglu_fp8(s["a"], s["a_scale"], s["offsets"], s["counts"], shape,
                                     s["w_gate_up"], s["s_gate_up"], s["w_down"], s["s_down"],
                                     expert_out=s["out"], workspace=ws)
    shape = moe.Shape(s["T"], s["H"], s["E"], s["k"], 1, 1, torch.bfloat16)
    ws = _workspace(s, lambda: moe.layer_workspace_bytes(shape, s["I"]))
    return moe.layer(s["logits"], s["x"], s["k"], s["w_gate_up"], s["w_down"],
                     s_gate_up=s["s_gate_up"], s_down=s["s_down"], y=s["y"], workspace=ws)


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
    if op == "quantize":
        n = case["batch"] * case["rows"] * case["cols"]
        blocks = case["batch"] * -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // 128)
        return {"bytes": n * (3 if case["dtype"] == "bf16" else 5) + 4 * blocks, "flops": 2 * n}
    T, E, k = case["T"], case["E"], case["k"]
    rows = T * k
    if op == "dispatch":
        H = case["H"]
        b = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * H * b + rows * (H + 4 * -(-H // 128) + 4), "flops": 2 * T * H}
    live = _live_experts(case)
    if op == "gemm":
        N, K = case["N"], case["K"]
        return {"bytes": rows * (K + K // 32 + 2 * N) + live * N * K, "flops": 2 * rows * N * K}
    H, I = case["H"], case["I"]
    flops = 6 * rows * H * I
    if op == "swiglu":
        return {"bytes": rows * (H + H // 32 + 2 * H) + live * 3 * H * I, "flops": flops}
    b = 2 if case["weights"] == "bf16" else 1
    return {"bytes": live * 3 * H * I * b + T * (4 * E + 4 * H) + rows * 8, "flops": flops}


# ------------------------------------------------------------------- exact

def _power_of_two(e):
    """2^e in 64 bits, from its bit pattern (pow and ldexp may be an ulp off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quantize(x, block_rows):
    """The same blocks from the definition: the scale from the binary exponent
    of amax / 448, each value to the nearest multiple of its binade's step."""
    x = x.double()
    B, R, C = x.shape
    q = torch.empty_like(x)
    scale = torch.empty(B, -(-R // block_rows), -(-C // 128), dtype=torch.float64, device=x.device)
    for j in range(scale.shape[2]):
        cols = x[:, :, 128 * j:128 * (j + 1)]
        if block_rows == 1:
            amax = cols.abs().amax(2)
        else:
            amax = torch.stack([cols[:, r:r + block_rows].abs().amax((1, 2))
                                for r in range(0, R, block_rows)], 1)
        f, e = torch.frexp(amax / 448.0)  # f in [0.5, 1): the power of two at or above
        s = _power_of_two(torch.where(f > 0.5, e, e - 1))
        s = torch.where(amax > 0, s.clamp(min=2.0 ** -126), 1.0)
        scale[:, :, j] = s
        v = cols / s.repeat_interleave(block_rows, 1)[:, :R, None]
        _, e = torch.frexp(v)
        step = _power_of_two((e - 1).clamp(min=-6) - 3)
        q[:, :, 128 * j:128 * (j + 1)] = torch.round(v / step) * step
    return q, scale


def _exact_scaled(q, scale, block_rows):
    """One matrix of 8-bit values as 64-bit numbers."""
    out = q.double()
    for j in range(scale.shape[1]):
        col = scale[:, j].double().repeat_interleave(block_rows)[:q.shape[0], None]
        out[:, 128 * j:128 * (j + 1)] *= col
    return out


def _exact_ffn(x, wg, wd, I, eight_bit_rows):
    gu = x @ wg.t()
    g, u = gu[:, :I], gu[:, I:]
    h = g * torch.sigmoid(g) * u
    if eight_bit_rows:
        hq, hs = _exact_quantize(h.unsqueeze(0), 1)
        h = _exact_scaled(hq[0], hs[0], 1)
    return h @ wd.t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s["x"], case["block_rows"])
    if op == "dispatch":
        q, scale = _exact_quantize(s["x"].unsqueeze(0), 1)
        send_q = torch.empty(s["send_q"].shape, dtype=torch.float64, device=_DEV)
        send_scale = torch.empty(s["send_scale"].shape, dtype=torch.float64, device=_DEV)
        for i in range(case["k"]):
            send_q[s["pos"][:, i].long()] = q[0]
            send_scale[s["pos"][:, i].long()] = scale[0]
        return send_q, send_scale
    if op in ("gemm", "swiglu"):
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=_DEV)
        for e, (n, o) in enumerate(zip(s["counts"].tolist(), s["offsets"].tolist())):
            if n == 0:
                continue
            a = _exact_scaled(s["a"][o:o + n], s["a_scale"][o:o + n], 1)
            if op == "gemm":
                out[o:o + n] = a @ _exact_scaled(s["w"][e], s["w_scale"][e], 128).t()
            else:
                out[o:o + n] = _exact_ffn(a, _exact_scaled(s["w_gate_up"][e], s["s_gate_up"][e], 128),
                                          _exact_scaled(s["w_down"][e], s["s_down"][e], 128),
                                          case["I"], True)
        return out
    k = case["k"]
    logits, x = s["logits"].double(), s["x"].double()
    T, E = logits.shape
    # highest logit first, the lower id where two are equal
    idx = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    gate = torch.softmax(torch.gather(logits, 1, idx), 1)
    y = torch.zeros(T, case["H"], dtype=torch.float64, device=_DEV)
    for e in range(E):
        token, place = torch.where(idx == e)
        if token.numel() == 0:
            continue
        wg, wd = s["w_gate_up"][e], s["w_down"][e]
        if case["weights"] == "fp8":
            wg = _exact_scaled(wg, s["s_gate_up"][e], 128)
            wd = _exact_scaled(wd, s["s_down"][e], 128)
        o = _exact_ffn(x[token], wg.double(), wd.double(), case["I"], False)
        y[token] += gate[token, place].unsqueeze(1) * o
    return y, idx.int(), gate
