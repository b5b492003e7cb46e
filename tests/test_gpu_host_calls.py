"""The C++ marshalling of the plain calls (wb_host) against the long way through ctypes (GPU): the same bits, and the same answers where a
call is not plain."""
import ctypes

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


def test_a_call_that_failed_is_not_made_again(wb, host):
    # a status other than a refusal may come from behind the call's first launch: gradients scaled once may not be scaled twice
    from whisper_encoder_gb300 import _lib
    lib, made = _lib.load(), []
    kinds = {n: ctypes.CFUNCTYPE(ctypes.c_int, *_lib.SIGNATURES[n][1]) for n in (
        "wb_cross_attention", "wb_cross_attention_backward", "wb_clip_grad_norm", "wb_policy_loss", "wb_policy_loss_backward")}

    def failing(name, status):
        return kinds[name](lambda *a: made.append(name) or status)

    q, k = torch.randn(2, 3, 128, device=DEV).bfloat16(), torch.randn(2, 5, 64, device=DEV).bfloat16()
    out, lse = wb.cross_attention(q, k, k)
    x, labels = torch.ones(4, 9, device=DEV), torch.zeros(4, 9, dtype=torch.int64, device=DEV)
    _, weight = wb.policy_loss(x, x, x, labels)
    calls = [("wb_cross_attention", lambda: wb.cross_attention(q, k, k)),
             ("wb_cross_attention_backward", lambda: wb.cross_attention_backward(out, q, k, k, out, lse)),
             ("wb_clip_grad_norm", lambda: wb.clip_grad_norm([x], 0.5)),
             ("wb_policy_loss", lambda: wb.policy_loss(x, x, x, labels)),
             ("wb_policy_loss_backward", lambda: wb.policy_loss_backward(x[0, :1], x, x, x, labels, weight))]
    try:
        for name, call in calls:
            for status in (_lib.WB_ECUDA, _lib.WB_ETIMEOUT, _lib.WB_EBOUNDS):
                fake = failing(name, status)
                _lib.bind_host(host, lib, {name: fake})
                made.clear()
                with pytest.raises(wb.WbError) as e:
                    call()
                assert made == [name] and name in str(e.value) and _lib.status_string(status) in str(e.value)
                assert bool((x == 1).all())
            # a refusal comes before anything is launched: the long way is taken, with its own checks and messages
            for status in (_lib.WB_EINVAL, _lib.WB_EUNSUPPORTED, _lib.WB_EWORKSPACE):
                fake = failing(name, status)
                _lib.bind_host(host, lib, {name: fake})
                made.clear()
                call()
                assert made == [name]
                x.fill_(1)
    finally:
        _lib.bind_host(host, lib)
    assert wb.check_device_error() == 0


def test_an_allocation_that_fails(wb, host):
    # a result of 16 GB (its rows are the same 1 GB for all items) in a process that may have 8
    q, k = torch.zeros(1, 1, 2048, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 5, 64, dtype=torch.bfloat16, device=DEV)
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(8 * 2 ** 30 / torch.cuda.mem_get_info()[1])
    try:
        rows = torch.zeros(1, 1 << 18, 2048, dtype=torch.bfloat16, device=DEV)
        with pytest.raises(torch.OutOfMemoryError):
            wb.cross_attention(rows.expand(16, -1, -1), k.expand(16, -1, -1), k.expand(16, -1, -1))
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert wb.cross_attention(q, k, k)[0].shape == q.shape and wb.check_device_error() == 0
