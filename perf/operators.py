"""The operators of the FFN blocks around the FP8 linears, as measured cases.

Three operators, each in its plain form (elementary torch operations in fp32,
run when `own` is false) and as the calls that a user makes of this package
(`own` true):

  linear_epilogue   FP8 W8A8 linear with bias, activation and residual:
                    Y = fp16(act((Xq . Wq^T) * s_x * s_w + bias) + residual)
  moe_route         router of a mixture of experts: the top-k experts of each
                    token from fp16 logits, their softmax weights, and the
                    expert-grouped row layout the grouped linears read
  moe_layer         a whole mixture-of-experts FFN for a few tokens: per-token
                    E4M3 quantization, expert up projection (optionally gated),
                    activation, E4M3 quantization of the hidden rows, expert
                    down projection, weighted sum over a token's experts, and
                    residual
"""
import math

import torch

own = False

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoded token through a square projection of the size sweep, everything in the epilogue
        {"name": "linear_m1", "op": "linear", "M": 1, "N": 4096, "K": 4096, "act": "silu", "bias": True,
         "residual": True, "x_fmt": "e4m3"},
        # a decode batch of 32 requests through the same projection
        {"name": "linear_m32", "op": "linear", "M": 32, "N": 4096, "K": 4096, "act": "gelu", "bias": True,
         "residual": False, "x_fmt": "e4m3"},
        # a ragged prefill of odd sizes with E5M2 activations (tiles cut on every side)
        {"name": "linear_ragged_e5m2", "op": "linear", "M": 333, "N": 1000, "K": 1040, "act": "gelu_tanh",
         "bias": True, "residual": True, "x_fmt": "e5m2"},
        # the up projection of the dense FFN pair: bias and GELU
        {"name": "linear_ffn_up", "op": "linear", "M": 8192, "N": 8192, "K": 2048, "act": "gelu", "bias": True,
         "residual": False, "x_fmt": "e4m3"},
        # its down projection: bias, and the block's input added back
        {"name": "linear_ffn_down", "op": "linear", "M": 8192, "N": 2048, "K": 8192, "act": "none", "bias": True,
         "residual": True, "x_fmt": "e4m3"},
        # routing one decoded token: latency
        {"name": "route_t1", "op": "route", "T": 1, "E": 64, "topk": 2, "renormalize": True, "masked": False},
        # an odd batch over many experts, some of them switched off (-inf logits), weights over all experts
        {"name": "route_t1000_masked", "op": "route", "T": 1000, "E": 160, "topk": 6, "renormalize": False,
         "masked": True},
        # the tokens of the full-size MoE layer
        {"name": "route_t8192", "op": "route", "T": 8192, "E": 64, "topk": 2, "renormalize": True, "masked": False},
        # one decoded token through the MoE FFN
        {"name": "moe_t1", "op": "moe", "T": 1, "E": 64, "topk": 2, "K": 2048, "F": 1024, "N": 2048, "act": "silu",
         "gated": False, "residual": True, "padded": 0},
        # eight tokens, gated experts
        {"name": "moe_t8_gated", "op": "moe", "T": 8, "E": 64, "topk": 4, "K": 2048, "F": 1024, "N": 2048,
         "act": "silu", "gated": True, "residual": False, "padded": 0},
        # a padded batch (three tokens without experts) of odd sizes
        {"name": "moe_t13_ragged", "op": "moe", "T": 13, "E": 20, "topk": 3, "K": 1040, "F": 272, "N": 1000,
         "act": "gelu", "gated": False, "residual": True, "padded": 3},
        # the largest batch of a few tokens: nearly every expert is read
        {"name": "moe_t64", "op": "moe", "T": 64, "E": 64, "topk": 2, "K": 2048, "F": 1024, "N": 2048, "act": "gelu",
         "gated": False, "residual": True, "padded": 0},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, -(-lo // step) * step), hi // step * step)


def draw(rng):
    op = rng.choice(("linear", "route", "moe"))
    if op == "linear":
        M, N, K = _spread(rng, 1, 8192), _spread(rng, 8, 8192, 8), _spread(rng, 16, 8192, 16)
        while M * N * K > 8192 * 8192 * 2048:
            M = max(1, M // 2)
        return {"op": op, "M": M, "N": N, "K": K, "act": rng.choice(ACTIVATIONS), "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.6, "x_fmt": rng.choice(("e4m3", "e4m3", "e5m2"))}
    if op == "route":
        E = _spread(rng, 2, 512)
        T = _spread(rng, 1, 8192)
        while T * E > 8192 * 64 * 4:
            T = max(1, T // 2)
        return {"op": op, "T": T, "E": E, "topk": rng.randint(1, min(8, E)), "renormalize": rng.random() < 0.5,
                "masked": rng.random() < 0.3}
    T, E = _spread(rng, 1, 64), _spread(rng, 2, 128)
    topk = rng.randint(1, min(8, E))
    gated = rng.random() < 0.5
    K, F, N = _spread(rng, 256, 4096, 16), _spread(rng, 128, 2048, 16), _spread(rng, 256, 4096, 8)
    while E * F * (K * (2 if gated else 1) + N) > 64 * 1024 * 4096:
        F = max(16, F // 32 * 16)
    while T * topk * F * (K * (2 if gated else 1) + N) > 64 * 8 * 1024 * 4096:
        T = max(1, T // 2)
    return {"op": op, "T": T, "E": E, "topk": topk, "K": K, "F": F, "N": N, "act": rng.choice(ACTIVATIONS),
            "gated": gated, "residual": rng.random() < 0.5, "padded": rng.choice((0, 0, T // 4))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


def _codes(x, fmt="e4m3"):
    """Per-row FP8 codes (uint8) and fp32 scales of x [..., K]."""
    dtype, top = FP8[fmt]
    a = x.float().abs().amax(-1, keepdim=True).clamp_min(1e-12)
    limit = torch.full_like(a, top)   # tensor by tensor: one rounded division, not a product with a reciprocal
    q = (x.float() * (limit / a)).clamp(-top, top).to(dtype)
    return q.view(torch.uint8), (a / limit).squeeze(-1).contiguous()


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """fp16 activations with a few outlier channels, as the path's tokens have."""
    x = _normal(g, M, K)
    ch = torch.randperm(K, generator=g, device="cuda")[:max(1, K // 200)]
    x[:, ch] *= 30.0
    return x.half()


def _expert_weights(g, E, N, K):
    q = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, N), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        q[e:e + n], s[e:e + n] = _codes((_normal(g, n, N, K) * 0.02).half())
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    st = {"case": dict(case)}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        st["Xq"], st["s_x"] = _codes(_activations(g, M, K), case["x_fmt"])
        st["Wq"], st["s_w"] = _codes((_normal(g, N, K) * 0.02).half())
        st["bias"] = (_normal(g, N) * 0.5).half() if case["bias"] else None
        st["residual"] = _normal(g, M, N).half() if case["residual"] else None
        return st
    T, E, k = case["T"], case["E"], case["topk"]
    logits = _normal(g, T, E).half()
    if case["op"] == "route":
        if case["masked"]:   # a third of the experts switched off, never all
            off = torch.randperm(E, generator=g, device="cuda")[:E // 3]
            logits[:, off] = float("-inf")
        st["logits"] = logits
        return st
    top = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    experts = top.indices[:, :k].to(torch.int32).contiguous()
    e = torch.exp(top.values[:, :k] - top.values[:, :1])
    st["weights"] = (e / e.sum(1, keepdim=True)).contiguous()
    if case["padded"]:
        experts[T - case["padded"]:] = -1
    st["experts"] = experts
    st["X"] = _activations(g, T, case["K"])
    st["Wq_up"], st["s_up"] = _expert_weights(g, E, case["F"] * (2 if case["gated"] else 1), case["K"])
    st["Wq_down"], st["s_down"] = _expert_weights(g, E, case["N"], case["F"])
    st["residual"] = _normal(g, T, case["N"]).half() if case["residual"] else None
    return st


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def run(st):
    c = st["case"]
    if own:
        import fp8_quantized_generative_b200 as fq
        if c["op"] == "linear":
            return fq.linear_epilogue(st["Xq"], st["s_x"], st["Wq"], st["s_w"], bias=st["bias"], activation=c["act"],
                                      residual=st["residual"], x_fmt=c["x_fmt"])
        if c["op"] == "route":
            r = fq.moe_route(st["logits"], c["topk"], renormalize=c["renormalize"])
            return {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "row_token": r.row_token,
                    "row_weight": r.row_weight, "token_rows": r.token_rows}
        return fq.moe_layer(st["X"], st["experts"], st["weights"], st["Wq_up"], st["s_up"], st["Wq_down"],
                            st["s_down"], activation=c["act"], gated=c["gated"], residual=st["residual"])
    if c["op"] == "linear":
        return _linear(st, c)
    if c["op"] == "route":
        return _route(st, c)
    return _moe(st, c)


def _act(z, name):
    if name == "relu":
        return torch.clamp_min(z, 0.0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _values(codes, fmt="e4m3"):
    return codes.view(FP8[fmt][0]).float()


def _linear(st, c):
    z = (_values(st["Xq"], c["x_fmt"]) @ _values(st["Wq"]).t()) * st["s_x"][:, None] * st["s_w"][None, :]
    if st["bias"] is not None:
        z = z + st["bias"].float()
    y = _act(z, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.half()


def _route(st, c):
    logits, k = st["logits"].float(), c["topk"]
    T, E = logits.shape
    top = torch.sort(logits, dim=1, descending=True, stable=True)   # ties: the lowest expert first
    experts = top.indices[:, :k]
    m = top.values[:, :1]
    e = torch.exp(top.values[:, :k] - m)
    weights = e / (e.sum(1, keepdim=True) if c["renormalize"] else torch.exp(logits - m).sum(1, keepdim=True))
    flat = experts.reshape(-1)
    place = torch.arange(T * k, device=logits.device)
    order = torch.argsort(flat * (T * k) + place)   # rows by (expert, token)
    counts = (flat[:, None] == torch.arange(E, device=logits.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    token_rows = torch.empty_like(order)
    token_rows[order] = place
    i32 = torch.int32
    return {"experts": experts.to(i32), "weights": weights, "offsets": offsets.to(i32),
            "row_token": torch.div(order, k, rounding_mode="floor").to(i32), "row_weight": weights.reshape(-1)[order],
            "token_rows": token_rows.reshape(T, k).to(i32)}


def _moe(st, c):
    T, k = st["experts"].shape
    xq, s_x = _codes(st["X"])
    used = (st["experts"] >= 0).reshape(-1)
    e = st["experts"].reshape(-1).clamp_min(0).long()
    x = _values(xq).repeat_interleave(k, 0)                                    # [T*k, K]
    z = torch.bmm(_values(st["Wq_up"][e]), x[:, :, None]).squeeze(-1)
    z = z * s_x.repeat_interleave(k)[:, None] * st["s_up"][e]
    if c["gated"]:
        h = _act(z[:, :c["F"]], c["act"]) * z[:, c["F"]:]
    else:
        h = _act(z, c["act"])
    hq, s_h = _codes(h.half())
    y = torch.bmm(_values(st["Wq_down"][e]), _values(hq)[:, :, None]).squeeze(-1)
    y = y * s_h[:, None] * st["s_down"][e]
    y = torch.where(used[:, None], y * st["weights"].reshape(-1)[:, None], torch.zeros_like(y))
    out = y.reshape(T, k, -1).sum(1)
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return out.half()


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        out = 2 * M * N * (2 if c["residual"] else 1) + (2 * N if c["bias"] else 0)
        return {"bytes": M * K + N * K + 4 * (M + N) + out, "flops": 2 * M * N * K}
    T, E, k = c["T"], c["E"], c["topk"]
    if c["op"] == "route":
        return {"bytes": 2 * T * E + 5 * 4 * T * k + 4 * (E + 1), "flops": 2 * T * E}
    live = T - c["padded"]
    up = c["F"] * (2 if c["gated"] else 1)
    read = E * (1.0 - (1.0 - k / E) ** live)   # experts that at least one token chose, on average
    per = up * c["K"] + c["N"] * c["F"] + 4 * (up + c["N"])
    io = 2 * T * c["K"] + 2 * T * c["N"] * (2 if c["residual"] else 1) + 8 * T * k
    return {"bytes": read * per + io, "flops": 2 * live * k * (up * c["K"] + c["N"] * c["F"])}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _table(fmt):
    """The 256 values of an FP8 format from its fields: sign, exponent, mantissa."""
    mant, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    v = []
    for code in range(256):
        e, f = (code & 127) >> mant, code & ((1 << mant) - 1)
        mag = math.ldexp(f, 1 - bias - mant) if e == 0 else math.ldexp((1 << mant) + f, e - bias - mant)
        v.append(-mag if code & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _act64(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":   # z times the normal distribution function
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def _quantized64(x16):
    """E4M3 values (float64) and scales of fp16 rows: one fp32 division for the
    multiplier and one for the scale, one fp32 product per value, then the
    nearest E4M3 value (ties to the even code)."""
    a = torch.clamp_min(x16.float().abs().amax(-1, keepdim=True), 1e-12)
    limit = torch.full_like(a, 448.0)
    v = (x16.float() * (limit / a)).double()
    size = v.abs().clamp(max=448.0)
    step = torch.pow(2.0, torch.clamp_min(torch.floor(torch.log2(size.clamp_min(1e-300))), -6.0) - 3.0)
    return torch.sign(v) * torch.clamp(torch.round(size / step) * step, max=448.0), (a / limit).double()


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "linear":
        x = _table(c["x_fmt"])[st["Xq"].int()] * st["s_x"].double()[:, None]
        w = _table("e4m3")[st["Wq"].int()] * st["s_w"].double()[:, None]
        z = torch.einsum("mk,nk->mn", x, w)
        if st["bias"] is not None:
            z += st["bias"].double()
        y = _act64(z, c["act"])
        return y if st["residual"] is None else y + st["residual"].double()
    if c["op"] == "route":
        l = st["logits"].double().cpu()
        T, E = l.shape
        k, rows = c["topk"], []
        experts, weights = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k, dtype=torch.float64)
        for t, line in enumerate(l.tolist()):
            best = sorted(range(E), key=lambda e: (-line[e], e))[:k]
            over = best if c["renormalize"] else range(E)
            total = math.fsum(math.exp(line[e] - line[best[0]]) for e in over)
            for j, e in enumerate(best):
                experts[t, j] = e
                weights[t, j] = math.exp(line[e] - line[best[0]]) / total
                rows.append((e, t, j))
        rows.sort()
        token_rows = torch.zeros(T, k, dtype=torch.int32)
        for r, (e, t, j) in enumerate(rows):
            token_rows[t, j] = r
        offsets = torch.zeros(E + 1, dtype=torch.int32)
        for e, _, _ in rows:
            offsets[e + 1] += 1
        return {"experts": experts, "weights": weights, "offsets": torch.cumsum(offsets, 0).to(torch.int32),
                "row_token": torch.tensor([t for _, t, _ in rows], dtype=torch.int32),
                "row_weight": torch.stack([weights[t, j] for _, t, j in rows]), "token_rows": token_rows}
    x, s_x = _quantized64(st["X"])
    x = x * s_x
    value = _table("e4m3")
    out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device="cuda")
    experts = st["experts"].cpu()
    for e in sorted(set(experts.reshape(-1).tolist()) - {-1}):
        at = (st["experts"] == e).nonzero()
        t, j = at[:, 0], at[:, 1]
        w = value[st["Wq_up"][e].int()] * st["s_up"][e].double()[:, None]
        z = x[t] @ w.t()
        h = _act64(z[:, :c["F"]], c["act"]) * z[:, c["F"]:] if c["gated"] else _act64(z, c["act"])
        h, s_h = _quantized64(h.half())
        w = value[st["Wq_down"][e].int()] * st["s_down"][e].double()[:, None]
        out.index_add_(0, t, (h * s_h) @ w.t() * st["weights"].double()[t, j][:, None])
    return out if st["residual"] is None else out + st["residual"].double()
