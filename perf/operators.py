"""Cases of the training operators: layer norm with its backward pass, softmax cross entropy over a
large vocabulary and distillation from a teacher's top logits, both straight from hidden states and the
projection matrix.

`run` computes them in their plain form (elementary torch operations in 32 bits, one rounding at the
end) or, with `own` set, by the framework's entry points.  `exact` gives the same outputs from the
operators' definitions in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ---------------------------------- cases ----------------------------------
def listed():
    return [
        # the last layer norm of a decoder that answers one token at a time
        {"name": "ln_fwd_token", "op": "ln", "dir": "fwd", "rows": 1, "d": 1280, "type": "bf16", "residual": True},
        # every position of a batch of 32 half-minute chunks, residual added in the same pass
        {"name": "ln_fwd_batch", "op": "ln", "dir": "fwd", "rows": 48000, "d": 1280, "type": "bf16", "residual": True},
        # the same batch on the way back, the residual branch's gradient added
        {"name": "ln_bwd_batch", "op": "ln", "dir": "bwd", "rows": 48000, "d": 1280, "type": "bf16", "residual": True},
        # both directions in 32 bits at a width that no vector load divides
        {"name": "ln_step_odd_f32", "op": "ln", "dir": "step", "rows": 4097, "d": 1283, "type": "f32", "residual": False},
        # both directions over an FFN's width in half precision
        {"name": "ln_step_wide_f16", "op": "ln", "dir": "step", "rows": 3001, "d": 5120, "type": "f16", "residual": True},
        # the log-probability of one token (rescoring a hypothesis as it grows)
        {"name": "ce_fwd_token", "op": "ce", "dir": "fwd", "m": 1, "d": 1280, "v": 51866, "padding": 0.0, "smoothing": 0.0},
        # validation loss over the transcripts of a few chunks
        {"name": "ce_fwd_eval", "op": "ce", "dir": "fwd", "m": 1500, "d": 1280, "v": 51866, "padding": 0.1, "smoothing": 0.0},
        # a training step of the vocabulary head: 32 transcripts padded to 448 tokens
        {"name": "ce_step_batch", "op": "ce", "dir": "step", "m": 14336, "d": 1280, "v": 51866, "padding": 0.25, "smoothing": 0.0},
        # a short transcript against a small model's head, odd sizes, smoothed labels
        {"name": "ce_step_short", "op": "ce", "dir": "step", "m": 77, "d": 384, "v": 51865, "padding": 0.0, "smoothing": 0.1},
        # how far a student is from its teacher on one transcript
        {"name": "distill_fwd_eval", "op": "distill", "dir": "fwd", "m": 448, "d": 1280, "v": 51866, "k": 100, "padding": 0.0,
         "temperature": 2.0},
        # a distillation step: 10 transcripts padded to 448 tokens, 64 stored logits a token
        {"name": "distill_step_batch", "op": "distill", "dir": "step", "m": 4480, "d": 1280, "v": 51866, "k": 64, "padding": 0.2,
         "temperature": 2.0},
        # a small student on a short transcript, few stored logits
        {"name": "distill_step_short", "op": "distill", "dir": "step", "m": 100, "d": 384, "v": 51865, "k": 8, "padding": 0.1,
         "temperature": 1.0},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ce", "distill"])
    if op == "ln":
        d = _log_uniform(rng, 64, 5120)
        if rng.random() < 0.7:
            d = max(64, d // 64 * 64)
        return {"op": op, "dir": rng.choice(["fwd", "bwd", "step"]), "rows": _log_uniform(rng, 1, min(48000, 48000 * 1280 // d)), "d": d,
                "type": rng.choice(["bf16", "f16", "f32"]), "residual": rng.random() < 0.5}
    case = {"op": op, "dir": rng.choice(["fwd", "step"]), "m": _log_uniform(rng, 1, 8000), "d": 8 * rng.randint(16, 160),
            "v": _log_uniform(rng, 1000, 51866), "padding": rng.choice([0.0, 0.1, 0.3])}
    if op == "ce":
        case["smoothing"] = rng.choice([0.0, 0.1])
    else:
        case["k"] = _log_uniform(rng, 1, 128)
        case["temperature"] = rng.choice([1.0, 2.0])
    return case


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    g = _generator(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if case["op"] == "ln":
        rows, d, t = case["rows"], case["d"], TYPES[case["type"]]
        # a residual stream: a few features far larger than the rest, a mean that is not zero
        scale = torch.exp(0.5 * normal(d))
        x = (normal(rows, d) * scale + 0.3).to(t)
        s = {"case": dict(case), "x": x, "g": 1 + 0.1 * normal(d), "b": 0.1 * normal(d),
             "res": normal(rows, d).to(t) if case["residual"] else None}
        if case["dir"] != "fwd":
            s["dy"] = (normal(rows, d) * 1e-2).to(t)
            s["dt"] = (normal(rows, d) * 1e-2).to(t) if case["residual"] else None
        if case["dir"] == "bwd":   # what the forward pass left behind
            s["res"] = None
            xf = x.float()
            mu = xf.mean(1)
            s["stats"] = torch.stack([mu, torch.rsqrt((xf - mu[:, None]).square().mean(1) + EPS)], 1).contiguous()
        return s
    m, d, v = case["m"], case["d"], case["v"]
    w = (0.05 * normal(v, d)).to(torch.bfloat16)
    first = torch.randint(0, v, (m,), generator=g, device=DEV)
    # hidden states that favour their token by a little or by a lot, as a trained head's do
    lean = 8 * torch.rand(m, generator=g, device=DEV) / (0.0025 * d)
    x = (normal(m, d) + lean[:, None] * w[first].float()).to(torch.bfloat16)
    pad = torch.rand(m, generator=g, device=DEV) < case["padding"]
    pad[0] = False
    s = {"case": dict(case), "x": x, "w": w, "dloss": torch.full((m,), 1.0 / int((~pad).sum()), device=DEV)}
    if case["op"] == "ce":
        s["labels"] = torch.where(pad, -100, first)
    else:
        k = case["k"]
        index = torch.randint(0, v, (m, k), generator=g, device=DEV)
        index[:, 0] = first
        s["index"] = torch.where(pad[:, None], -1, index)
        top = 10 - torch.empty((m, k), device=DEV).exponential_(0.3, generator=g)
        s["top"] = top.sort(1, descending=True).values.contiguous()
    return s


# ------------------------------- plain forms -------------------------------
def _plain_ln(s):
    case, t = s["case"], s["x"].dtype
    out = {}
    x = s["x"]
    if case["dir"] == "bwd":
        total, mu, rs = x, s["stats"][:, 0], s["stats"][:, 1]
    else:
        total = x if s["res"] is None else (x.float() + s["res"].float()).to(t)
        tf = total.float()
        mu = tf.mean(1)
        rs = torch.rsqrt((tf - mu[:, None]).square().mean(1) + EPS)
        out["y"] = ((tf - mu[:, None]) * rs[:, None] * s["g"] + s["b"]).to(t)
        out["total"] = total
        out["stats"] = torch.stack([mu, rs], 1)
    if case["dir"] != "fwd":
        h = (total.float() - mu[:, None]) * rs[:, None]
        dy = s["dy"].float()
        u = dy * s["g"]
        dx = rs[:, None] * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
        if s["dt"] is not None:
            dx = dx + s["dt"].float()
        out.update(dx=dx.to(t), dg=(dy * h).sum(0), db=dy.sum(0))
    return out


def _plain_head(s, scale, target, valid, const):
    """Row statistics of the scaled logits and, for a step, the gradients; `target`: dense, `const`: sum t log t."""
    x = torch.where(valid[:, None], s["x"], 0).float()
    w = s["w"].float()
    logits = (x @ w.T) * scale
    top = logits.amax(1, keepdim=True)
    lse = (top + (logits - top).exp().sum(1, keepdim=True).log())[:, 0]
    kl = (const + lse - (target * logits).sum(1)) / scale ** 2
    out = {"loss": torch.where(valid, kl, 0.0), "lse": torch.where(valid, lse, 0.0)}
    if s["case"]["dir"] == "step":
        dlogits = ((logits - lse[:, None]).exp() - target) * torch.where(valid, s["dloss"] / scale, 0.0)[:, None]
        out["dx"] = (dlogits @ w).to(torch.bfloat16)
        out["dw"] = (dlogits.T @ x).to(torch.bfloat16)
    return out


def _plain_ce(s):
    labels, v, e = s["labels"], s["case"]["v"], s["case"]["smoothing"]
    valid = labels >= 0
    target = torch.full((labels.numel(), v), e / v, device=DEV)
    target.scatter_add_(1, labels.clamp(min=0)[:, None], torch.full_like(labels, 1.0 - e, dtype=torch.float32)[:, None])
    return _plain_head(s, 1.0, target, valid, 0.0)


def _plain_distill(s):
    index, case = s["index"], s["case"]
    there = index >= 0
    valid = there.any(1)
    t = torch.where(there, s["top"].float() / case["temperature"], -math.inf)
    p = (t - torch.where(valid, t.amax(1), 0.0)[:, None]).exp()
    p = p / torch.where(valid, p.sum(1), 1.0)[:, None]
    target = torch.zeros((index.shape[0], case["v"]), device=DEV).scatter_add_(1, index.clamp(min=0), p)
    const = (target * target.clamp(min=1e-38).log()).sum(1)
    return _plain_head(s, 1.0 / case["temperature"], target, valid, const)


# ------------------------------ the framework ------------------------------
def _own(s):
    import whisper_encoder_gb300 as wb
    case = s["case"]
    step = case["dir"] == "step"
    if case["op"] == "ln":
        out, total, stats = {}, s["x"], s.get("stats")
        if case["dir"] != "bwd":
            y, total, stats = wb.layernorm_forward(s["x"], s["g"], s["b"], EPS, residual=s["res"])
            out.update(y=y, total=total, stats=stats)
        if case["dir"] != "fwd":
            dx, dg, db = wb.layernorm_backward(s["dy"], total, s["g"], stats, dtotal=s["dt"])
            out.update(dx=dx, dg=dg, db=db)
        return out
    if case["op"] == "ce":
        loss, lse = wb.linear_cross_entropy(s["x"], s["w"], s["labels"], case["smoothing"])
        out = {"loss": loss, "lse": lse}
        if step:
            out["dx"], out["dw"] = wb.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["labels"], lse, case["smoothing"])
        return out
    loss, lse = wb.linear_distill(s["x"], s["w"], s["top"], s["index"], case["temperature"])
    out = {"loss": loss, "lse": lse}
    if step:
        out["dx"], out["dw"] = wb.linear_distill_backward(s["dloss"], s["x"], s["w"], s["top"], s["index"], lse, case["temperature"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"ln": _plain_ln, "ce": _plain_ce, "distill": _plain_distill}[state["case"]["op"]](state)


# ----------------------------------- work ----------------------------------
def work(case):
    if case["op"] == "ln":
        n, size = case["rows"] * case["d"], TYPES[case["type"]].itemsize
        tensors = 0
        if case["dir"] != "bwd":
            tensors += 2 + (2 if case["residual"] else 0)
        if case["dir"] != "fwd":
            # a step reads the rows that it normalised again for the way back only where they do not fit on the chip
            tensors += (3 if case["dir"] == "bwd" else 2) + (1 if case["residual"] else 0)
        return {"bytes": n * size * tensors + 8 * case["rows"] + 16 * case["d"], "flops": 8 * n}
    m, d, v = case["m"], case["d"], case["v"]
    n = m - int(case["padding"] * m)
    moved = 2 * (n * d + v * d) + 8 * m * (1 + (12 * case["k"] // 8 if case["op"] == "distill" else 1))
    products = 1
    if case["dir"] == "step":
        products, moved = 3, moved + 2 * (m * d + v * d)
    return {"bytes": moved, "flops": 2 * n * d * v * products}


# ----------------------------------- exact ---------------------------------
def _exact_ln(s):
    case, t = s["case"], s["x"].dtype
    x, g, b = s["x"].double(), s["g"].double(), s["b"].double()
    d = x.shape[1]
    out = {}
    if case["dir"] == "bwd":
        mu, rs = s["stats"].double().unbind(1)
    else:
        if s["res"] is not None:   # the stored sum is what is normalised
            x = (x + s["res"].double()).to(t).double()
        mu = x.sum(1) / d
        rs = 1 / ((x - mu[:, None]).pow(2).sum(1) / d + EPS).sqrt()
        out = {"y": torch.addcmul(b, (x - mu[:, None]) * rs[:, None], g), "total": x, "stats": torch.stack([mu, rs], 1)}
    if case["dir"] == "fwd":
        return out
    dy = s["dy"].double()
    hat = (x - mu[:, None]) * rs[:, None]
    gy = g * dy
    along = torch.einsum("rd,rd->r", gy, hat) / d
    dx = (gy - gy.sum(1)[:, None] / d - along[:, None] * hat) * rs[:, None]
    out["dx"] = dx if s["dt"] is None else dx + s["dt"].double()
    out["dg"] = torch.einsum("rd,rd->d", dy, hat)
    out["db"] = torch.einsum("rd->d", dy)
    return out


def _exact_head(s):
    case = s["case"]
    m, d = s["x"].shape
    v = s["w"].shape[0]
    w = s["w"].double()
    temperature, smooth = case.get("temperature", 1.0), case.get("smoothing", 0.0)
    loss, lse = torch.zeros(m, device=DEV, dtype=torch.float64), torch.zeros(m, device=DEV, dtype=torch.float64)
    step = case["dir"] == "step"
    dx = torch.zeros((m, d), device=DEV, dtype=torch.float64)
    dw = torch.zeros((v, d), device=DEV, dtype=torch.float64)
    kept = (s["labels"] if case["op"] == "ce" else s["index"][:, 0]).ge(0).nonzero()[:, 0]
    for rows in kept.split(2048):
        x = s["x"][rows].double()
        log_q = torch.log_softmax((x @ w.T) / temperature, 1)
        at = torch.arange(rows.numel(), device=DEV)
        first = x @ w[0] / temperature
        lse[rows] = first - log_q[:, 0]
        if case["op"] == "ce":
            y = s["labels"][rows]
            loss[rows] = -(1 - smooth) * log_q[at, y] - smooth * log_q.sum(1) / v
            grad = log_q.exp() - smooth / v
            grad[at, y] -= 1 - smooth
        else:
            p = torch.softmax(s["top"][rows].double() / temperature, 1)
            goal = torch.zeros_like(log_q)
            goal.index_put_((at[:, None].expand_as(p), s["index"][rows]), p, accumulate=True)
            loss[rows] = temperature ** 2 * torch.special.xlogy(goal, goal).sub_(goal * log_q).sum(1)
            grad = (log_q.exp() - goal) * temperature
        if step:
            grad *= s["dloss"][rows].double()[:, None]
            dx[rows] = grad @ w
            dw += grad.T @ x
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw} if step else {"loss": loss, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_ln(s) if case["op"] == "ln" else _exact_head(s)
