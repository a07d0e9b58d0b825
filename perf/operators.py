"""The operators around the W4A4 linear that are measured: the norms of a block, routing, and the
mixture-of-experts layer for a few tokens.

``own`` picks the side: False runs each operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), True makes the package's calls.  ``exact`` says what the results
are in 64 bits.

norm   what stands between two blocks:  h' = h + s * gate * post(y),  n = pre(h')
route  router logits -> the k experts of each token, their weights, and the rows sorted by expert
       for the grouped linear
moe    y[t] = sum_j w[t,j] * W2_e . act(Wg_e x[t]) * (Wu_e x[t]),  e = ids[t,j], every product W4A4
       MXFP4 with the package's channel factors and block-32 Hadamard rotation
"""
import math

import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # decoding one token: nothing but latency
        {"name": "norm 1x2048", "op": "norm", "rows": 1, "width": 2048, "residual": "bf16", "gate": "none", "post": True},
        # a small batch of image tokens, a gate of its own for each token, a width that is no power of two
        {"name": "norm 77x5120", "op": "norm", "rows": 77, "width": 5120, "residual": "bf16", "gate": "token", "post": False},
        # a prefill of the dense workloads' length, a learned residual scale for each channel
        {"name": "norm 4096x1024", "op": "norm", "rows": 4096, "width": 1024, "residual": "bf16", "gate": "channel", "post": True},
        # long prefill with the residual stream in fp32, one gate for each sequence, a ragged last one
        {"name": "norm 16385x2048 fp32", "op": "norm", "rows": 16385, "width": 2048, "residual": "fp32", "gate": "sequence", "post": True},
        # routing of one decoded token
        {"name": "route 1x128", "op": "route", "tokens": 1, "experts": 128, "k": 8, "logits": "fp32", "score": "softmax", "renorm": True},
        # a ragged batch, experts that do not fill a warp's lanes evenly, sigmoid scores
        {"name": "route 1001x60", "op": "route", "tokens": 1001, "experts": 60, "k": 4, "logits": "fp32", "score": "sigmoid", "renorm": False},
        # routing in front of the grouped workload: 8192 tokens over 128 experts
        {"name": "route 8192x128", "op": "route", "tokens": 8192, "experts": 128, "k": 8, "logits": "bf16", "score": "softmax", "renorm": True},
        # decoding one token of the 128-expert layer: eight experts' weights are all there is to read
        {"name": "moe 1 of 128", "op": "moe", "tokens": 1, "experts": 128, "k": 8, "hidden": 2048, "inner": 768, "act": "silu", "score": "softmax", "renorm": True},
        # a few users of a small layer, gated by GELU
        {"name": "moe 5 of 16", "op": "moe", "tokens": 5, "experts": 16, "k": 2, "hidden": 1024, "inner": 512, "act": "gelu", "score": "sigmoid", "renorm": True},
        # a decoding batch of 16: most of its experts have one or two rows
        {"name": "moe 16 of 128", "op": "moe", "tokens": 16, "experts": 128, "k": 8, "hidden": 2048, "inner": 768, "act": "silu", "score": "softmax", "renorm": True},
        # the largest batch that still counts as few: every expert is read once
        {"name": "moe 128 of 128", "op": "moe", "tokens": 128, "experts": 128, "k": 8, "hidden": 2048, "inner": 768, "act": "silu", "score": "softmax", "renorm": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "moe", "moe"])
    if op == "norm":
        width = 16 * _log_int(rng, 4, 512)
        return {"op": op, "rows": _log_int(rng, 1, min(16385, 16385 * 2048 // width)), "width": width,
                "residual": rng.choice(["bf16", "fp32"]), "gate": rng.choice(["none", "token", "channel", "sequence"]),
                "post": rng.random() < 0.7}
    score = rng.choice(["softmax", "sigmoid"])
    if op == "route":
        experts = _log_int(rng, 4, 512)
        return {"op": op, "tokens": _log_int(rng, 1, min(8192, 8192 * 128 // experts)), "experts": experts,
                "k": rng.randint(1, min(8, experts)), "logits": rng.choice(["bf16", "fp32"]), "score": score,
                "renorm": rng.random() < 0.5}
    hidden, inner = 256 * _log_int(rng, 1, 16), 256 * _log_int(rng, 1, 8)
    experts = _log_int(rng, 2, max(2, min(128, 128 * 2048 * 768 // (hidden * inner))))
    return {"op": op, "tokens": _log_int(rng, 1, 128), "experts": experts, "k": rng.randint(1, min(8, experts)),
            "hidden": hidden, "inner": inner, "act": rng.choice(["silu", "gelu"]), "score": score,
            "renorm": rng.random() < 0.5}


def work(case):
    if case["op"] == "norm":
        m, c = case["rows"], case["width"]
        h = 4 if case["residual"] == "fp32" else 2
        gate_rows = {"none": 0, "token": m, "channel": 1, "sequence": -(-m // _sequence(m))}[case["gate"]]
        weights = 4 * c * (2 if case["post"] else 1)
        return {"bytes": m * c * (2 * h + 2 + 2) + 2 * gate_rows * c + weights, "flops": 10 * m * c}
    t, e, k = case["tokens"], case["experts"], case["k"]
    if case["op"] == "route":
        return {"bytes": t * e * (4 if case["logits"] == "fp32" else 2) + t * k * 12 + 8 * e, "flops": 4 * t * e}
    hidden, inner = case["hidden"], case["inner"]
    read = e * (1 - (1 - k / e) ** t)  # experts that at least one token picks, on average
    per_expert = 3 * hidden * inner * 17 / 32 + 4 * (hidden + inner)
    return {"bytes": read * per_expert + t * hidden * 4 + t * e * 4, "flops": 6 * t * k * hidden * inner}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _sequence(rows):
    """Rows of a sequence where each has a gate of its own: about eight sequences, the last one ragged."""
    return max(1, rows // 8)


def _inputs(case, seed):
    """The tensors of a case that both sides and exact() start from."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        m, c = case["rows"], case["width"]
        h = 4 * normal(m, c)
        h[:, torch.randperm(c, generator=g, device="cuda")[: max(1, c // 100)]] *= 20  # a few loud channels
        gate_rows = {"none": 0, "token": m, "channel": 1, "sequence": -(-m // _sequence(m))}[case["gate"]]
        return {
            "h": h if case["residual"] == "fp32" else h.bfloat16(),
            "y": (2 * normal(m, c)).bfloat16(),
            "w_post": 1 + 0.2 * normal(c) if case["post"] else None,
            "gate": (0.5 + 0.3 * normal(gate_rows, c)).bfloat16() if gate_rows else None,
            "rows_per_gate": {"token": 1, "sequence": _sequence(m)}.get(case["gate"], m),
            "w_pre": 1 + 0.2 * normal(c),
            "scale": 0.22,
        }
    t, e = case["tokens"], case["experts"]
    logits = 1.5 * normal(t, e)
    if case["op"] == "route":
        return {"logits": logits if case["logits"] == "fp32" else logits.bfloat16()}
    hidden, inner = case["hidden"], case["inner"]
    x = normal(t, hidden)
    x[:, torch.randperm(hidden, generator=g, device="cuda")[: max(1, hidden // 100)]] *= 20
    w_up = 0.02 * normal(e, 2 * inner, hidden)  # gate rows, then up rows
    w_down = 0.02 * normal(e, hidden, inner)
    # channel factors as a calibration run over more tokens would leave them
    d_up = (x.abs().amax(0).clamp_min(1.0) / w_up.abs().amax(1)).sqrt().clamp(1e-2, 1e2)
    loud = torch.rand(inner, generator=g, device="cuda") + 0.25
    d_down = (loud / w_down.abs().amax(1)).sqrt().clamp(1e-2, 1e2)
    return {"x": x.bfloat16(), "logits": logits, "w_up": w_up, "w_down": w_down, "d_up": d_up, "d_down": d_down}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "moe":  # weights are quantised once, offline
        w_up, w_down = s.pop("w_up"), s.pop("w_down")
        if own:
            import w4a4_mxfp4_quantize_b200 as mq

            s["up"] = mq.prepare_gate_up(w_up, s["d_up"])
            s["down"] = mq.prepare_weights(w_down, s["d_down"])
        else:
            s["up"] = _quantize(_rotate(w_up * s["d_up"][:, None, :]))
            s["down"] = _quantize(_rotate(w_down * s["d_down"][:, None, :]))
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "moe": _own_moe}[case["op"]](case, state)
    return {"norm": _plain_norm, "route": _plain_route, "moe": _plain_moe}[case["op"]](case, state)


def _own_norm(case, s):
    import w4a4_mxfp4_quantize_b200 as mq

    return mq.block_norm(s["h"], s["y"], w_post=s["w_post"], gate=s["gate"], rows_per_gate=s["rows_per_gate"],
                         w_pre=s["w_pre"], scale=s["scale"], eps=EPS)


def _own_route(case, s):
    import w4a4_mxfp4_quantize_b200 as mq

    score = mq.SCORE_SOFTMAX if case["score"] == "softmax" else mq.SCORE_SIGMOID
    return mq.moe_route(s["logits"], case["k"], score=score, renorm=case["renorm"])


def _own_moe(case, s):
    import w4a4_mxfp4_quantize_b200 as mq

    score = mq.SCORE_SOFTMAX if case["score"] == "softmax" else mq.SCORE_SIGMOID
    act = mq.ACT_SILU if case["act"] == "silu" else mq.ACT_GELU_TANH
    return mq.moe_mm(s["x"], s["logits"], s["d_up"], *s["up"], s["d_down"], *s["down"], inner=case["inner"],
                     k=case["k"], score=score, renorm=case["renorm"], act_type=act)


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _rms(v, w):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w


def _plain_norm(case, s):
    branch = s["y"].float()
    if s["w_post"] is not None:
        branch = _rms(branch, s["w_post"])
    if s["gate"] is not None:
        rows = torch.arange(case["rows"], device=branch.device) // s["rows_per_gate"]
        branch = branch * s["gate"].float()[rows]
    h = (s["h"].float() + s["scale"] * branch).to(s["h"].dtype)
    return h, _rms(h.float(), s["w_pre"]).bfloat16()


def _choose(logits, k, score, renorm):
    """The k largest logits of each row, ties to the lowest index, and their weights."""
    logits = logits.float()
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-top))
        w = s / s.sum(-1, keepdim=True) if renorm else s
    else:
        p = torch.exp(top - top[:, :1])
        total = p.sum(-1, keepdim=True) if renorm else torch.exp(logits - top[:, :1]).sum(-1, keepdim=True)
        w = p / total
    return ids, w


def _plain_route(case, s):
    ids, w = _choose(s["logits"], case["k"], case["score"], case["renorm"])
    flat = ids.reshape(-1)
    counts = torch.zeros(case["experts"], dtype=torch.int64, device=flat.device)
    counts.scatter_add_(0, flat, torch.ones_like(flat))
    order = torch.sort(flat, stable=True).indices
    return ids.int(), w, counts, order.int()


def _rotate(v):
    """Block-32 Sylvester Hadamard rotation along the last axis, stage by stage."""
    shape = v.shape
    for h in (1, 2, 4, 8, 16):
        v = v.reshape(*shape[:-1], -1, 2, h)
        v = torch.stack((v[..., 0, :] + v[..., 1, :], v[..., 0, :] - v[..., 1, :]), -2)
    return v.reshape(shape)


def _power(e):
    """2**e of whole numbers in [-126, 127], exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantize(v):
    """MXFP4 along the last axis: packed E2M1 codes (nearest, ties to even, saturating) and E8M0 scales."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    exponent = (torch.frexp(b.abs().amax(-1)).exponent - 3).clamp_min(-126)
    q = b * _power(-exponent[..., None])
    mag = q.abs().clamp_max(6.0)
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    mag = torch.round(mag / step) * step
    index = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
    code = (index + 8 * (q < 0).to(torch.uint8)).reshape(*v.shape[:-1], -1, 2)
    return code[..., 0] + 16 * code[..., 1], (exponent + 127).to(torch.uint8)


def _decode(codes, scales):
    value = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1, 32)
    return (value[pair.int()] * _power(scales[..., None].int() - 127)).flatten(-2)


def _linear(x, d, weights):
    """x [A, T, K] bf16 values in fp32, d [A, K], weights (codes, scales) of [A, N, K] -> [A, T, N] in fp32."""
    u = _rotate((x * (1 / d)[:, None, :]).bfloat16().float()).bfloat16().float()
    return torch.bmm(_decode(*_quantize(u)), _decode(*weights).transpose(1, 2)) / 32


def _plain_moe(case, s):
    ids, w = _choose(s["logits"], case["k"], case["score"], case["renorm"])
    active = torch.unique(ids)  # the experts that some token picked
    share = torch.zeros_like(s["logits"]).scatter_(1, ids, w)[:, active].t()  # [A, T]
    x = s["x"].float().expand(len(active), -1, -1)
    gate, up = _linear(x, s["d_up"][active], [v[active] for v in s["up"]]).chunk(2, -1)
    if case["act"] == "silu":
        gate = gate / (1 + torch.exp(-gate))
    else:
        gate = 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate**3)))
    inner = (gate * up).bfloat16().float()
    y = _linear(inner, s["d_down"][active], [v[active] for v in s["down"]])
    return (share[..., None] * y).sum(0).bfloat16()


# ---------------------------------------------------------------------------------------------
# what the results are, in 64 bits
# ---------------------------------------------------------------------------------------------
def _power_below(v):
    """The largest power of two that is not above v > 0, by clearing the fraction's bits."""
    return (v.view(torch.int64) & (0x7FF << 52)).view(torch.float64)


def _round_bf16(v):
    """float64 -> the nearest value of bfloat16's grid, ties to even, still float64."""
    step = _power_below(v.abs().clamp_min(2.0**-126)) / 128
    return torch.round(v / step) * step


def _hadamard(device):
    i = torch.arange(32, device=device)
    bits = (i[:, None] & i[None, :]).unsqueeze(-1) >> torch.arange(5, device=device) & 1
    return (1 - 2 * (bits.sum(-1) % 2)).double()


def _mx_value(v):
    """The values that MXFP4 codes of v stand for: the nearest entry of the table in each block's scale."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    scale = _power_below(amax.clamp_min(2.0**-124)) / 4
    table = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    between = (table[1:] + table[:-1]) / 2
    mag = (b / scale).abs()
    low = torch.bucketize(mag, between)  # a value on a border gets the lower entry ...
    high = torch.bucketize(mag, between, right=True)  # ... or the upper one; the even code is right
    index = torch.where(low % 2 == 0, low, high)
    return (table[index] * torch.sign(b) * scale).flatten(-2)


def _exact_expert(x, d, w):
    """One expert's linear: x [T, K], d [K] fp32, w [N, K] fp32 -> [T, N] in 64 bits."""
    had = _hadamard(x.device)
    scaled = _round_bf16((x.float() * (1 / d)).double())  # the definition multiplies by the rounded reciprocal
    u = _round_bf16((scaled.unflatten(-1, (-1, 32)) @ had).flatten(-2))
    t = (((w * d).double().unflatten(-1, (-1, 32))) @ had).flatten(-2).float().double()
    return _mx_value(u) @ _mx_value(t).t() / 32


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        y = s["y"].double()
        if s["w_post"] is not None:
            y = y / torch.sqrt(y.square().mean(1, keepdim=True) + EPS) * s["w_post"].double()
        if s["gate"] is not None:
            y = y * torch.repeat_interleave(s["gate"].double(), s["rows_per_gate"], 0)[: case["rows"]]
        h = s["h"].double() + s["scale"] * y
        h_out = h.to(s["h"].dtype).double()
        return h_out, h_out / torch.sqrt(h_out.square().mean(1, keepdim=True) + EPS) * s["w_pre"].double()
    logits = s["logits"].double()
    # the rank of a logit: how many go before it
    n = torch.arange(case["experts"], device=logits.device)
    ids = torch.empty(len(logits), case["k"], dtype=torch.int64, device=logits.device)
    for i in range(0, len(logits), 256):
        a = logits[i : i + 256]
        before = (a[:, None, :] > a[:, :, None]) | ((a[:, None, :] == a[:, :, None]) & (n[None, :] < n[:, None]))
        rank = before.sum(-1)
        ids[i : i + 256] = torch.argsort(rank, 1)[:, : case["k"]]
    score = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if case["op"] == "route":
        return None, w, None, None
    out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=logits.device)
    for e in range(case["experts"]):
        token, at = torch.nonzero(ids == e, as_tuple=True)
        if not len(token):
            continue
        both = _exact_expert(s["x"][token], s["d_up"][e], s["w_up"][e])
        gate, up = both[:, : case["inner"]], both[:, case["inner"] :]
        if case["act"] == "silu":
            gate = gate * torch.sigmoid(gate)
        else:
            gate = gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate.pow(3)))
        inner = _round_bf16(gate * up)
        y = _exact_expert(inner, s["d_down"][e], s["w_down"][e])
        out.index_add_(0, token, w[token, at][:, None] * y)
    return out
