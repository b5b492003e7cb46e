"""The C++ marshalling of the plain calls (wb_host) against the long way through ctypes (GPU): the same bits, and the same answers where a
call is not plain."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture
def host(wb):
    from whisper_encoder_gb300 import _lib
    h = _lib.host_calls()
    assert h, "wb_host.so is not built: every call takes the long way"
    return h


def _everything(wb):
    g = torch.Generator(device=DEV).manual_seed(1)
    q, do = (torch.randn(3, 70, 256, device=DEV, generator=g).bfloat16() for _ in range(2))
    kv = torch.randn(3, 200, 256, device=DEV, generator=g).bfloat16()
    k, v = kv[..., :128], kv[..., 128:]
    lens = torch.tensor([200, 0, 77], dtype=torch.int32, device=DEV)
    out = []
    for kw in ({}, {"kv_lens": lens}, {"q_lens": lens, "scale": 1}):
        o, lse = wb.cross_attention(q, k, v, **kw)
        out += [o, lse, *wb.cross_attention_backward(do, q, k, v, o, lse, **kw),
                *wb.cross_attention_backward(do, q, k, v, o, lse, need_dq=0, **kw)[1:], wb.cross_attention_backward(do, q, k, v, o, lse, need_dkv=False, **kw)[0]]
    grads = [torch.randn(n, device=DEV, generator=g).to(t) for n in (5, 0, 9000) for t in (torch.bfloat16, torch.float16, torch.float32)]
    wide = [torch.empty(t.shape, device=DEV) for t in grads]
    out += [wb.grad_norm(grads), wb.clip_grad_norm(grads, 2.0, out=wide), *wide, wb.clip_grad_norm(tuple(grads), 2), *grads]
    nll = torch.rand(300, 40, device=DEV, generator=g)
    labels = torch.randint(-1, 5, (300, 40), device=DEV, generator=g)
    for S in (300, 7):
        for adv in (torch.randn(S, device=DEV, generator=g), torch.randn(S, 40, device=DEV, generator=g)):
            for ref, beta in ((None, 0.0), (nll[:S] - 0.1, 0.3)):
                a = (nll[:S], nll[:S] + 0.2, adv, labels[:S])
                stats, weight = wb.policy_loss(*a, ref_nll=ref, kl_weight=beta, per_sequence=S == 7)
                out += [stats, weight, wb.policy_loss_backward(torch.full((1,), 2.0, device=DEV), *a, weight, ref_nll=ref, kl_weight=beta)]
    assert wb.check_device_error() == 0
    return out


def test_the_same_bits(wb, host, monkeypatch):
    from whisper_encoder_gb300 import _lib
    fast = _everything(wb)
    monkeypatch.setattr(_lib, "_HOST", False)
    slow = _everything(wb)
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device and not a.requires_grad
        assert torch.equal(a, b)


def test_plain_calls_take_the_short_way_and_others_do_not(wb, host):
    q, k = torch.zeros(2, 3, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 5, 64, dtype=torch.bfloat16, device=DEV)
    x, labels = torch.zeros(4, 9, device=DEV), torch.zeros(4, 9, dtype=torch.int64, device=DEV)
    assert host.cross_attention(q, k, k, 0.125, None, None) is not None
    assert host.clip_grad_norm([x], 1.0, None) is not None
    assert host.policy_loss(x, x, x[:, 0].contiguous(), labels, None, 0.2, 0.2, 0.0, False) is not None
    for bad in ((q.cpu(), k, k, 0.125, None, None), (q, k, k, 0.0, None, None), (q, k, k, "a", None, None), (q, k[:1], k[:1], 0.125, None, None),
                (q.float(), k, k, 0.125, None, None), (q, k, k, 0.125, labels[0], None), (q, None, k, 0.125, None, None), (q,)):
        assert host.cross_attention(*bad) is None
    assert host.clip_grad_norm([x, x], 1.0, [x, x]) is None and host.clip_grad_norm([x], -1.0, [x]) is None
    assert host.clip_grad_norm([], 1.0, None) is None and host.clip_grad_norm([x.T], 1.0, None) is None
    assert host.policy_loss(x, x, x, labels, None, 0.2, 0.2, 0.5, False) is None            # a KL term without a reference
    assert host.policy_loss_backward(x, x, x, x, labels, x[:, 0], None, 0.2, 0.2, 0.0) is None
    assert wb.check_device_error() == 0


def test_outputs_on_a_side_stream_and_in_a_graph(wb, host):
    q, k = torch.randn(2, 30, 128, device=DEV).bfloat16(), torch.randn(2, 50, 64, device=DEV).bfloat16()
    want = wb.cross_attention(q, k, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = wb.cross_attention(q, k, k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = wb.cross_attention(q, k, k)
    graph.replay()
    with torch.inference_mode():
        quiet = wb.cross_attention(q, k, k)
    for a, b, c, d in zip(want, got, inside, quiet):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
