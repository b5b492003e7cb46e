"""One training step of a decoder's reader behind the encoder, by the entry points in a row (GPU): norm, query projection, cross
attention to the encoder's states over cross_kv, output projection on the residual stream, vocabulary head, clipped policy loss,
the way back and clipped gradients, against float64 autograd of the same step.

How far: a gradient passes at most 16 roundings to bf16 (y, q, p, out, residual stream, softmax - target, x', and on the way back
dr, dout, dS, dq / dk / dv, dy and its own) of 2^-8 of a value each.  On its way through the softmax a rounding of q or k is multiplied by a
score: a sum of 64 products, each off by its own rounding, is off as a 2-norm by 2^-8 of the scores' root mean square, which
stays below 2.  As 2-norms of independent errors: 2 sqrt(16) 2^-8."""
import pytest
import torch

import synthetic

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOUND = 2 * 16 ** 0.5 * 2.0 ** -8


def _leaves(d, V, g):
    n = lambda *s, k=0.05: torch.randn(*s, device=DEV, generator=g) * k  # noqa: E731
    return {"wq": n(d, d).bfloat16(), "wkv": n(2 * d, d).bfloat16(), "bkv": n(2 * d), "wo": n(d, d).bfloat16(), "head": n(V, d).bfloat16(),
            "gamma": 1 + n(d), "beta": n(d)}


def test_one_step(wb):
    dims = synthetic.TINY
    d, V, B, T = dims.d_model, 1001, 3, 60
    g = torch.Generator(device=DEV).manual_seed(4)
    w = _leaves(d, V, g)
    enc = torch.randn(B, 1500, d, device=DEV, generator=g).bfloat16()
    h = torch.randn(B, T, d, device=DEV, generator=g).bfloat16()
    labels = torch.randint(0, V, (B, T), device=DEV, generator=g)
    q_lens = torch.tensor([T, 41, 17], dtype=torch.int32, device=DEV)
    kv_lens = torch.tensor([1500, 900, 0], dtype=torch.int32, device=DEV)          # one recording without sound
    labels = torch.where(torch.arange(T, device=DEV) < q_lens[:, None], labels, -100)
    adv = torch.tensor([0.7, -1.1, 0.4], device=DEV)

    kv = wb.cross_kv(enc, dims, [(w["wkv"], w["bkv"])])[0].view(B, 1500, 2 * d)
    k, v = kv[..., :d], kv[..., d:]
    y, total, stats = wb.layernorm_forward(h, w["gamma"], w["beta"])
    q = wb.linear(y.view(-1, d), w["wq"]).view(B, T, d)
    out, lse = wb.cross_attention(q, k, v, q_lens=q_lens, kv_lens=kv_lens)
    r = wb.linear(out.view(-1, d), w["wo"], resid=h.view(-1, d))
    nll, lse_head = wb.linear_cross_entropy(r, w["head"], labels.view(-1))
    old, ref = nll.view(B, T) + 0.05, nll.view(B, T) - 0.1
    kw = dict(ref_nll=ref, clip_low=0.2, clip_high=0.2, kl_weight=0.2)
    loss, weight = wb.policy_loss(nll.view(B, T), old, adv, labels, per_sequence=True, **kw)

    dnll = wb.policy_loss_backward(torch.ones((), device=DEV), nll.view(B, T), old, adv, labels, weight, **kw)
    dr, d_head = wb.linear_cross_entropy_backward(dnll.view(-1), r, w["head"], labels.view(-1), lse_head)
    dq, dk, dv = wb.cross_attention_backward((dr @ w["wo"]).view(B, T, d), q, k, v, out, lse, q_lens=q_lens, kv_lens=kv_lens)
    dh, d_gamma, d_beta = wb.layernorm_backward((dq.view(-1, d) @ w["wq"]).view(B, T, d), total, w["gamma"], stats, dtotal=dr.view(B, T, d))
    dkv = torch.cat([dk, dv], 2).view(-1, 2 * d)
    grads = {"wq": dq.view(-1, d).mT @ y.view(-1, d), "wkv": dkv.mT @ enc.view(-1, d), "wo": dr.mT @ out.view(-1, d), "head": d_head,
             "gamma": d_gamma, "beta": d_beta}
    whole = {n: t.double() for n, t in grads.items()}
    norm = wb.clip_grad_norm(list(grads.values()), 1e-3)
    assert wb.check_device_error() == 0

    p = {n: t.double().requires_grad_() for n, t in w.items()}
    h64 = h.double().requires_grad_()
    kv64 = enc.double() @ p["wkv"].T + p["bkv"]
    y64 = torch.nn.functional.layer_norm(h64, (d,), p["gamma"], p["beta"], 1e-5)
    heads = lambda t: t.reshape(B, -1, dims.n_heads, 64).transpose(1, 2)  # noqa: E731
    s = heads(y64 @ p["wq"].T) @ heads(kv64[..., :d]).mT / 8
    there = (torch.arange(1500, device=DEV) < kv_lens[:, None])[:, None, None]
    s = s.masked_fill(~there, -1e300)
    assert float(s.detach().masked_fill(~there, 0).square().mean().sqrt()) < 2
    a = torch.softmax(s, -1) * there
    r64 = h64 + (a @ heads(kv64[..., d:])).transpose(1, 2).reshape(B, T, d) @ p["wo"].T
    on = labels >= 0
    nll64 = torch.nn.functional.cross_entropy((r64 @ p["head"].T).view(-1, V), labels.view(-1), reduction="none", ignore_index=-100).view(B, T)
    # the old and reference values are the kernels' own: constants of the step
    ratio = torch.exp(old.double() - nll64)
    free, held = ratio * adv.double()[:, None], ratio.clamp(0.8, 1.2) * adv.double()[:, None]
    x = nll64 - ref.double()
    token = -torch.minimum(free, held) + 0.2 * (torch.exp(x) - x - 1)
    want = (torch.where(on, token, 0.0).sum(1) / on.sum(1)).mean()
    want.backward()

    assert abs(float(loss[0]) - float(want.detach())) < BOUND * float(token.detach()[on].abs().mean())
    for n, t in whole.items():
        ref64 = p[n].grad
        assert float((t - ref64).norm() / ref64.norm()) < BOUND, n
    assert float((dh.double() - h64.grad).norm() / h64.grad.norm()) < BOUND
    total64 = torch.sqrt(sum(p[n].grad.square().sum() for n in grads))
    assert abs(float(norm) / float(total64) - 1) < BOUND and float(norm) > 1e-3
    for n, t in grads.items():                       # scaled in place: half a step of its type, and the factor's error
        off = (2.0 ** -8 if t.dtype == torch.bfloat16 else 2.0 ** -22) + 2.0 ** -18
        scaled = whole[n] * 1e-3 / float(norm)
        assert bool(((t.double() - scaled).abs() <= off * scaled.abs() + 1e-38).all()), n
