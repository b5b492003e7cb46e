"""Cases of the operators of a decoder that reads the encoder: cross attention (forward for many rows, for single
tokens and beams, and its backward pass), the global gradient norm with clipping, and a clipped policy loss
on the head's log-probabilities.

`run` computes them in their plain form (elementary torch operations in 32 bits, one rounding at the
end) or, with `own` set, by the framework's entry points.  `exact` gives the same outputs from the
operators' definitions in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
HEAD = 64                     # width of a head everywhere in this framework
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CLIP_LOW, CLIP_HIGH = 0.2, 0.28


# ---------------------------------- cases ----------------------------------
def listed():
    return [
        # one token of one hypothesis reads one half-minute chunk
        {"name": "cross_token", "op": "cross", "dir": "fwd", "s": 1, "tq": 1, "tk": 1500, "heads": 20, "kv_heads": 20, "ragged": False},
        # a step of a beam search: 5 hypotheses of each of 32 chunks
        {"name": "cross_beams", "op": "cross", "dir": "fwd", "s": 32, "tq": 5, "tk": 1500, "heads": 20, "kv_heads": 20, "ragged": False},
        # the prompt of one long recording's joined windows, heads that share keys and values
        {"name": "cross_long", "op": "cross", "dir": "fwd", "s": 1, "tq": 224, "tk": 13501, "heads": 16, "kv_heads": 4, "ragged": False},
        # scoring 32 transcripts of 448 tokens
        {"name": "cross_fwd_batch", "op": "cross", "dir": "fwd", "s": 32, "tq": 448, "tk": 1500, "heads": 20, "kv_heads": 20, "ragged": False},
        # a training step over the same batch, transcripts and recordings of different lengths
        {"name": "cross_step_batch", "op": "cross", "dir": "step", "s": 32, "tq": 448, "tk": 1500, "heads": 20, "kv_heads": 20,
         "ragged": True},
        # a small model's step on three short transcripts
        {"name": "cross_step_short", "op": "cross", "dir": "step", "s": 3, "tq": 77, "tk": 1371, "heads": 6, "kv_heads": 6, "ragged": True},
        # gradient norm of the whole encoder (monitoring)
        {"name": "norm_encoder", "op": "clip", "dir": "norm", "layers": 32, "d": 1280, "ffn": 5120, "type": "bf16", "max_norm": 1.0},
        # a vocabulary head and the layers next to it, clipped into 32 bits for the optimiser
        {"name": "clip_decoder", "op": "clip", "dir": "clip", "layers": 4, "d": 1280, "ffn": 5120, "type": "bf16", "max_norm": 0.5},
        # a small model's gradients, odd sizes
        {"name": "clip_small", "op": "clip", "dir": "clip", "layers": 2, "d": 387, "ffn": 1536, "type": "f32", "max_norm": 1.0},
        # sampled transcripts of a few chunks
        {"name": "policy_short", "op": "policy", "dir": "step", "s": 8, "t": 77, "kl": 0.05, "per_sequence": False},
        # 16 samples of each of 64 chunks
        {"name": "policy_batch", "op": "policy", "dir": "step", "s": 1024, "t": 448, "kl": 0.05, "per_sequence": True},
        # the loss alone over a large pool of samples, no KL term
        {"name": "policy_pool", "op": "policy", "dir": "fwd", "s": 16001, "t": 448, "kl": 0.0, "per_sequence": False},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "clip", "policy"])
    if op == "cross":
        kv_heads = rng.choice([1, 2, 4, 6, 8, 12, 16, 20])
        heads = kv_heads * rng.choice([1, 1, 1, 2, 4])
        tk = _log_uniform(rng, 1, 15000)
        tq = rng.choice([1, rng.randint(1, 16), _log_uniform(rng, 1, 448)])
        # no more scores, keys and queries than the largest listed case
        most = min(32 * 448 * 1500 * 20 // (tq * tk * heads), 32 * 1500 * 20 // (tk * kv_heads), 32 * 448 * 20 // (tq * heads))
        return {"op": op, "dir": rng.choice(["fwd", "step"]), "s": _log_uniform(rng, 1, max(1, min(64, most))), "tq": tq, "tk": tk,
                "heads": heads, "kv_heads": kv_heads, "ragged": rng.random() < 0.5}
    if op == "clip":
        d = rng.randint(64, 1280)
        layers = _log_uniform(rng, 1, min(24, 8 * 1280 ** 2 // d ** 2))
        return {"op": op, "dir": rng.choice(["norm", "clip"]), "layers": layers, "d": d, "ffn": 4 * d,
                "type": rng.choice(["bf16", "f16", "f32"]), "max_norm": rng.choice([0.5, 1.0, 1e6])}
    s = _log_uniform(rng, 1, 16000)
    return {"op": op, "dir": rng.choice(["fwd", "step"]), "s": s, "t": _log_uniform(rng, 1, min(2000, 16000 * 448 // s)),
            "kl": rng.choice([0.0, 0.05]), "per_sequence": rng.random() < 0.5}


def _clip_shapes(case):
    """Weights of a pre-norm layer (projections, feed-forward, norms, biases) `layers` times, as they lie."""
    d, f = case["d"], case["ffn"]
    return [(3 * d, d), (3 * d,), (d, d), (d,), (f, d), (f,), (d, f), (d,), (d,), (d,)] * case["layers"]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if case["op"] == "cross":
        s, tq, tk, h, hk = (case[n] for n in ("s", "tq", "tk", "heads", "kv_heads"))
        # keys and values side by side, as the projections of the encoder's states leave them
        kv = normal(s, tk, 2 * hk * HEAD).to(torch.bfloat16)
        # queries from flat to sharp: scores of a deviation between 0.3 and 4
        lean = 0.3 + 3.7 * torch.rand((s, tq, 1), generator=g, device=DEV)
        state = {"case": dict(case), "q": (normal(s, tq, h * HEAD) * lean).to(torch.bfloat16), "kv": kv,
                 "q_lens": None, "kv_lens": None}
        if case["ragged"]:
            state["q_lens"] = torch.randint(tq // 2, tq + 1, (s,), generator=g, device=DEV, dtype=torch.int32)
            state["kv_lens"] = torch.randint(tk // 2, tk + 1, (s,), generator=g, device=DEV, dtype=torch.int32)
            if s > 2:
                state["kv_lens"][1] = 0          # a recording without sound
        if case["dir"] == "step":
            state["dout"] = (1e-3 * normal(s, tq, h * HEAD)).to(torch.bfloat16)
        return state
    if case["op"] == "clip":
        shapes = _clip_shapes(case)
        t = TYPES[case["type"]]
        # matrices in the model's type, vectors (biases, norms) in 32 bits; layers of different size
        grads = [(normal(*shape) * (1e-3 * (1 + i % 7))).to(t if len(shape) > 1 else torch.float32) for i, shape in enumerate(shapes)]
        state = {"case": dict(case), "grads": grads}
        if case["dir"] == "clip":
            state["out"] = [torch.empty(x.shape, device=DEV) for x in grads]
        return state
    s, t = case["s"], case["t"]
    nll = torch.empty((s, t), device=DEV).exponential_(1.0, generator=g)
    lengths = torch.randint(0, t + 1, (s, 1), generator=g, device=DEV)
    lengths[0] = t
    labels = torch.randint(0, 51866, (s, t), generator=g, device=DEV)
    labels = torch.where(torch.arange(t, device=DEV) < lengths, labels, -100)
    return {"case": dict(case), "nll": nll, "old": nll + 0.2 * normal(s, t), "labels": labels,
            "ref": nll + 0.3 * normal(s, t) if case["kl"] else None, "advantage": normal(s),
            "dloss": torch.ones((), device=DEV)}


# ------------------------------- plain forms -------------------------------
def _plain_cross(s):
    case = s["case"]
    n, tq, tk, h, hk = (case[i] for i in ("s", "tq", "tk", "heads", "kv_heads"))
    kv = s["kv"].float().view(n, tk, 2, hk, HEAD).permute(2, 0, 3, 1, 4)
    k, v = kv[0][:, :, None], kv[1][:, :, None]                       # [s, hk, 1, tk, 64]

    def rows(x):                                                      # [s, tq, 64 h] -> [s, hk, g, tq, 64]
        return x.float().view(n, tq, hk, h // hk, HEAD).permute(0, 2, 3, 1, 4)

    def flat(x):
        return x.permute(0, 3, 1, 2, 4).reshape(n, tq, h * HEAD).to(torch.bfloat16)

    kv_ok, q_ok = None, None
    if s["kv_lens"] is not None:
        kv_ok = (torch.arange(tk, device=DEV) < s["kv_lens"][:, None])[:, None, None, None, :]
        q_ok = (torch.arange(tq, device=DEV) < s["q_lens"][:, None])[:, None, None, :, None]
        k = torch.where(kv_ok.mT, k, 0.0)
        v = torch.where(kv_ok.mT, v, 0.0)
    q = rows(s["q"])
    scores = (q @ k.mT) * HEAD ** -0.5
    if kv_ok is not None:
        scores = torch.where(kv_ok & q_ok, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    lse = top + total.log()
    p = p / torch.where(total > 0, total, 1.0)
    out = {"out": flat(p @ v), "lse": lse.reshape(n, h, tq)}
    if case["dir"] == "step":
        do = rows(s["dout"])
        if q_ok is not None:
            q, do = torch.where(q_ok, q, 0.0), torch.where(q_ok, do, 0.0)
        dp = do @ v.mT
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * HEAD ** -0.5
        out["dq"] = flat(ds @ k)
        for name, x in (("dk", ds.mT @ q), ("dv", p.mT @ do)):        # summed over the heads that share them
            out[name] = x.sum(2).permute(0, 2, 1, 3).reshape(n, tk, hk * HEAD).to(torch.bfloat16)
    return out


def _plain_clip(s):
    case = s["case"]
    norm = torch.stack([x.float().square().sum() for x in s["grads"]]).double().sum().sqrt()
    if case["dir"] == "norm":
        return {"norm": norm.float()}
    scale = torch.where(norm > case["max_norm"], case["max_norm"] / norm, 1.0).float()
    return {"norm": norm.float(), "grads": [x.float() * scale for x in s["grads"]]}


def _weights(labels, per_sequence):
    there = (labels >= 0).double().sum(1)
    if per_sequence:
        return torch.where(there > 0, 1 / (there.clamp(min=1) * (there > 0).sum().clamp(min=1)), 0.0)
    return torch.full_like(there, 1.0) / there.sum().clamp(min=1)


def _plain_policy(s):
    case = s["case"]
    there = s["labels"] >= 0
    weight = _weights(s["labels"], case["per_sequence"]).float()[:, None]
    a = s["advantage"][:, None]
    diff = s["old"].double() - s["nll"].double()                       # next to the border of the clip 32 bits are short
    clipped = torch.where(a > 0, diff > math.log1p(CLIP_HIGH), (diff < math.log1p(-CLIP_LOW)) & (a < 0))
    r = diff.float().exp()
    held = torch.where(a > 0, 1 + CLIP_HIGH, 1 - CLIP_LOW)
    loss = -torch.where(clipped, held, r) * a
    dnll = torch.where(clipped, 0.0, r * a)
    kl = torch.zeros_like(loss)
    if s["ref"] is not None:
        x = s["nll"].double() - s["ref"].double()
        kl = (x.expm1() - x).float()                                   # a difference that is x^2 / 2 for small x
        loss = loss + case["kl"] * kl
        dnll = dnll + case["kl"] * x.expm1().float()
    sums = [torch.where(there, weight * i, 0.0).double().sum().float() for i in (loss, kl, clipped.float())]
    out = {"stats": torch.stack(sums)}
    if case["dir"] == "step":
        out["dnll"] = torch.where(there, dnll * weight * s["dloss"], 0.0)
    return out


# ------------------------------ the framework ------------------------------
def _own(s):
    import whisper_encoder_gb300 as wb
    case = s["case"]
    if case["op"] == "cross":
        half = case["kv_heads"] * HEAD
        k, v = s["kv"][..., :half], s["kv"][..., half:]
        out, lse = wb.cross_attention(s["q"], k, v, q_lens=s["q_lens"], kv_lens=s["kv_lens"])
        result = {"out": out, "lse": lse}
        if case["dir"] == "step":
            result["dq"], result["dk"], result["dv"] = wb.cross_attention_backward(s["dout"], s["q"], k, v, out, lse, q_lens=s["q_lens"],
                                                                                   kv_lens=s["kv_lens"])
        return result
    if case["op"] == "clip":
        if case["dir"] == "norm":
            return {"norm": wb.grad_norm(s["grads"])}
        return {"norm": wb.clip_grad_norm(s["grads"], case["max_norm"], out=s["out"]), "grads": s["out"]}
    kwargs = dict(ref_nll=s["ref"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_weight=case["kl"])
    stats, weight = wb.policy_loss(s["nll"], s["old"], s["advantage"], s["labels"], per_sequence=case["per_sequence"], **kwargs)
    out = {"stats": stats}
    if case["dir"] == "step":
        out["dnll"] = wb.policy_loss_backward(s["dloss"], s["nll"], s["old"], s["advantage"], s["labels"], weight, **kwargs)
    return out


def run(state):
    if own:
        return _own(state)
    return {"cross": _plain_cross, "clip": _plain_clip, "policy": _plain_policy}[state["case"]["op"]](state)


# ----------------------------------- work ----------------------------------
def work(case):
    if case["op"] == "cross":
        s, tq, tk, h, hk = (case[n] for n in ("s", "tq", "tk", "heads", "kv_heads"))
        share = 0.75 if case["ragged"] else 1.0      # mean length of a ragged axis
        q, kv, lse = 2 * s * tq * h * HEAD, 4 * s * tk * hk * HEAD, 4 * s * tq * h
        products = 2
        moved = share * q + q + share * kv + lse
        if case["dir"] == "step":
            # dout read, dq, dk and dv written; q, k, v and out read once for both directions
            products, moved = 7, moved + share * q + q + kv
        return {"bytes": moved, "flops": 2 * products * s * h * tq * tk * HEAD * share * share}
    if case["op"] == "clip":
        size = TYPES[case["type"]].itemsize
        moved = flops = 0
        for shape in _clip_shapes(case):
            n = math.prod(shape)
            moved += n * ((size if len(shape) > 1 else 4) + (4 if case["dir"] == "clip" else 0))
            flops += 2 * n
        return {"bytes": moved, "flops": flops}
    n = case["s"] * case["t"]
    words = 4 + (1 if case["kl"] else 0) + (1 if case["dir"] == "step" else 0)
    return {"bytes": 4 * n * words + 4 * case["s"], "flops": 20 * n}


# ----------------------------------- exact ---------------------------------
def _exact_cross(s):
    case = s["case"]
    n, tq, tk, h, hk = (case[i] for i in ("s", "tq", "tk", "heads", "kv_heads"))
    group, step = h // hk, case["dir"] == "step"
    f64 = dict(device=DEV, dtype=torch.float64)
    res = {"out": torch.zeros((n, tq, h, HEAD), **f64), "lse": torch.full((n, h, tq), -math.inf, **f64)}
    if step:
        res.update(dq=torch.zeros((n, tq, h, HEAD), **f64), dk=torch.zeros((n, tk, hk, HEAD), **f64), dv=torch.zeros((n, tk, hk, HEAD), **f64))
    q_lens = [tq] * n if s["q_lens"] is None else s["q_lens"].tolist()
    kv_lens = [tk] * n if s["kv_lens"] is None else s["kv_lens"].tolist()
    for i in range(n):
        a, b = q_lens[i], kv_lens[i]
        if not a or not b:
            continue
        keys = s["kv"][i, :b].double().reshape(b, 2, hk, HEAD)
        k = keys[:, 0].repeat_interleave(group, 1)                    # one key head for each query head
        v = keys[:, 1].repeat_interleave(group, 1)
        q = s["q"][i, :a].double().reshape(a, h, HEAD)
        score = torch.einsum("qhe,khe->hqk", q, k) / math.sqrt(HEAD)
        lse = torch.logsumexp(score, 2)
        p = torch.exp(score - lse[:, :, None])
        res["lse"][i, :, :a] = lse
        o = torch.einsum("hqk,khe->qhe", p, v)
        res["out"][i, :a] = o
        if step:
            do = s["dout"][i, :a].double().reshape(a, h, HEAD)
            ds = p * (torch.einsum("qhe,khe->hqk", do, v) - torch.einsum("qhe,qhe->hq", do, o)[:, :, None]) / math.sqrt(HEAD)
            res["dq"][i, :a] = torch.einsum("hqk,khe->qhe", ds, k)
            res["dk"][i, :b] = torch.einsum("hqk,qhe->khe", ds, q).reshape(b, hk, group, HEAD).sum(2)
            res["dv"][i, :b] = torch.einsum("hqk,qhe->khe", p, do).reshape(b, hk, group, HEAD).sum(2)
    return {name: x if name == "lse" else x.flatten(2) for name, x in res.items()}


def _exact_policy(s):
    case = s["case"]
    stats = torch.zeros(3, device=DEV, dtype=torch.float64)
    counts = s["labels"].ge(0).sum(1).double()
    spoken = counts.gt(0).sum().double()
    dnll = torch.zeros(s["nll"].shape, device=DEV, dtype=torch.float64)
    for at in torch.arange(counts.numel(), device=DEV).split(2048):
        rows, cols = s["labels"][at].ge(0).nonzero(as_tuple=True)
        rows = rows + at[0]
        w = 1 / (counts[rows] * spoken) if case["per_sequence"] else torch.ones_like(rows, dtype=torch.float64) / counts.sum()
        nll, a = s["nll"][rows, cols].double(), s["advantage"][rows].double()
        ratio = torch.exp(s["old"][rows, cols].double() - nll)
        free, held = ratio * a, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * a
        token, grad = -torch.minimum(free, held), torch.where(free <= held, free, 0.0)
        stats[2] += (w * (held < free)).sum()
        if s["ref"] is not None:
            x = nll - s["ref"][rows, cols].double()
            k3 = torch.exp(x) - x - 1
            token, grad = token + case["kl"] * k3, grad + case["kl"] * (torch.exp(x) - 1)
            stats[1] += (w * k3).sum()
        stats[0] += (w * token).sum()
        dnll[rows, cols] = w * grad * s["dloss"].double()
    return {"stats": stats, "dnll": dnll} if case["dir"] == "step" else {"stats": stats}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "cross":
        return _exact_cross(s)
    if case["op"] == "policy":
        return _exact_policy(s)
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(x, dtype=torch.float64)) ** 2 for x in s["grads"]))
    value = torch.tensor(norm, device=DEV, dtype=torch.float64)
    if case["dir"] == "norm":
        return {"norm": value}
    ratio = min(1.0, case["max_norm"] / norm)
    return {"norm": value, "grads": [x.double() * ratio for x in s["grads"]]}
