"""The training operators in the bounds-checked debug build, between guard bytes, at sizes that pass 32
bits, from two streams at once and in a first call that is captured (GPU)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from test_gpu_debug import Guarded, _run_both, _stream, libs  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731


@pytest.mark.parametrize("rows,d,kind", [(129, 384, "bf16"), (1, 1280, "f16"), (301, 1283, "f32"), (77, 2568, "bf16"), (5, 5128, "f16"),
                                         (3, 10240, "f32"), (40, 7, "bf16"), (2000, 1280, "bf16")])
@pytest.mark.parametrize("residual", [False, True])
def test_layernorm_train(libs, rows, d, kind, residual):  # noqa: F811
    from whisper_encoder_gb300 import _lib as L
    t, ty = {"bf16": (torch.bfloat16, L.WB_BF16), "f16": (torch.float16, L.WB_F16), "f32": (torch.float32, L.WB_F32)}[kind]
    g = torch.Generator(device=DEV).manual_seed(rows)
    x, r, dy, dt = (torch.randn(rows, d, device=DEV, generator=g).to(t) for _ in range(4))
    gam, bet = (torch.randn(d, device=DEV, generator=g) for _ in range(2))

    def fn(lib):
        y, tot, st = Guarded((rows, d), t), Guarded((rows, d), t), Guarded((rows, 2), torch.float32)
        assert lib.wb_layernorm_forward(P(x), P(r) if residual else None, P(gam), P(bet), rows, d, 1e-5, ty, y.p,
                                        tot.p if residual else None, st.p, _stream()) == 0
        dx, dg, db = Guarded((rows, d), t), Guarded((d,), torch.float32), Guarded((d,), torch.float32)
        ws = Guarded((lib.wb_layernorm_backward_workspace_bytes(rows, d, ty),), torch.uint8)
        assert lib.wb_layernorm_backward(P(dy), tot.p if residual else P(x), P(gam), st.p, P(dt) if residual else None, rows, d, ty,
                                         dx.p, dg.p, db.p, ws.p, ws.n, _stream()) == 0
        torch.cuda.synchronize()
        assert ws.guards_intact()
        return [y, st, dx, dg, db] + ([tot] if residual else [])
    _run_both(libs, fn)


@pytest.mark.parametrize("M,d,V,k", [(1, 72, 333, 3), (16, 1288, 700, 9), (77, 384, 1001, 5), (129, 64, 2049, 17), (300, 776, 999, 40),
                                     (700, 136, 5003, 2)])
def test_head_losses(libs, M, d, V, k):  # noqa: F811
    from whisper_encoder_gb300 import _lib as L
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn(M, d, device=DEV, generator=g).to(torch.bfloat16)
    w = (torch.randn(V, d, device=DEV, generator=g) * 0.1).to(torch.bfloat16)
    labels = torch.randint(0, V, (M,), device=DEV, generator=g)
    labels[1::3] = -1
    index = torch.randint(-1, V, (M, k), device=DEV, generator=g)
    top = torch.randn(M, k, device=DEV, generator=g)
    dloss = torch.rand(M, device=DEV, generator=g)

    def fn(lib):
        out = []
        for ce in (True, False):
            query = lib.wb_linear_cross_entropy_workspace_bytes if ce else lib.wb_linear_distill_workspace_bytes
            back = lib.wb_linear_cross_entropy_backward_workspace_bytes if ce else lib.wb_linear_distill_backward_workspace_bytes
            shape = (M, d, V) if ce else (M, d, V, k)
            loss, lse = Guarded((M,), torch.float32), Guarded((M,), torch.float32)
            ws, wsb = Guarded((query(*shape),), torch.uint8), Guarded((back(*shape),), torch.uint8)
            dx, dw = Guarded((M, d), torch.bfloat16), Guarded((V, d), torch.bfloat16)
            if ce:
                assert lib.wb_linear_cross_entropy(P(x), P(w), P(labels), M, d, V, 0.1, loss.p, lse.p, ws.p, ws.n, _stream()) == 0
                assert lib.wb_linear_cross_entropy_backward(P(dloss), P(x), P(w), P(labels), lse.p, M, d, V, 0.1, dx.p, dw.p, wsb.p,
                                                            wsb.n, _stream()) == 0
            else:
                assert lib.wb_linear_distill(P(x), P(w), P(top), L.WB_F32, P(index), M, d, V, k, 2.0, loss.p, lse.p, ws.p, ws.n,
                                             _stream()) == 0
                assert lib.wb_linear_distill_backward(P(dloss), P(x), P(w), P(top), L.WB_F32, P(index), lse.p, M, d, V, k, 2.0, dx.p,
                                                      dw.p, wsb.p, wsb.n, _stream()) == 0
            torch.cuda.synchronize()
            assert ws.guards_intact() and wsb.guards_intact()
            out += [loss, lse, dx, dw]
        return out
    _run_both(libs, fn)


def test_layernorm_offsets_past_32_bits(wb):
    # more than 2^31 elements a tensor: the last rows against the same rows alone
    rows, d = (1 << 31) // 1280 + 1000, 1280
    x = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV)
    dy = torch.empty_like(x)
    for t in (x, dy):
        for i in range(0, rows, 1 << 18):
            t[i:i + (1 << 18)].normal_()
    g, b = torch.rand(d, device=DEV), torch.rand(d, device=DEV)
    y, total, stats = wb.layernorm_forward(x, g, b)
    dx, dg, db = wb.layernorm_backward(dy, total, g, stats)
    tail = slice(rows - 1500, rows)
    y2, total2, stats2 = wb.layernorm_forward(x[tail], g, b)
    dx2, _, _ = wb.layernorm_backward(dy[tail], total2, g, stats2)
    assert torch.equal(y[tail], y2) and torch.equal(stats[tail], stats2) and torch.equal(dx[tail], dx2)
    want = torch.zeros(d, dtype=torch.float64, device=DEV)
    for i in range(0, rows, 1 << 17):
        want += dy[i:i + (1 << 17)].double().sum(0)
    # sums of n terms of size about 1, rounded at the size of the sum, which grows as sqrt(n)
    assert float((db.double() - want).abs().max()) < 2.0 ** -24 * rows ** 0.5 * 4 * 152
    assert wb.check_device_error() == 0


@pytest.mark.parametrize("M", [3, 150])
def test_vocabulary_offsets_past_32_bits(wb, M):
    V, d = 2_300_000, 1024                              # w has 2.36e9 elements
    g = torch.Generator(device=DEV).manual_seed(5)
    w = torch.empty(V, d, dtype=torch.bfloat16, device=DEV)
    for i in range(0, V, 1 << 18):
        w[i:i + (1 << 18)].normal_(std=0.05, generator=g)
    x = torch.randn(M, d, device=DEV, generator=g).to(torch.bfloat16)
    labels = torch.randint(V - 200_000, V, (M,), device=DEV, generator=g)
    dloss = torch.ones(M, device=DEV)
    loss, lse = wb.linear_cross_entropy(x, w, labels)
    dx, dw = wb.linear_cross_entropy_backward(dloss, x, w, labels, lse)
    assert wb.check_device_error() == 0
    s = torch.cat([x.double() @ w[i:i + (1 << 17)].double().T for i in range(0, V, 1 << 17)], 1)
    ref = torch.logsumexp(s, 1)
    torch.testing.assert_close(lse.double(), ref, rtol=2 ** -20, atol=0)
    torch.testing.assert_close(loss.double(), ref - s.gather(1, labels[:, None])[:, 0], rtol=2 ** -18, atol=2 ** -18)
    D = torch.exp(s - ref[:, None])
    D.scatter_add_(1, labels[:, None], torch.full_like(D[:, :1], -1.0))
    for lo, hi in ((0, 1000), (V - 200_000, V)):
        want = D[:, lo:hi].T @ x.double()
        rel = float((dw[lo:hi].double() - want).norm() / want.norm())
        assert rel < 2.0 ** -8, rel                      # D and dw rounded to bf16, rms 2^-8 / sqrt(3) each


def test_two_calls_at_once(wb):
    M, d, V = 600, 512, 9000
    g = torch.Generator(device=DEV).manual_seed(6)
    cases = []
    for _ in range(2):
        x = torch.randn(M, d, device=DEV, generator=g).to(torch.bfloat16)
        w = (torch.randn(V, d, device=DEV, generator=g) * 0.1).to(torch.bfloat16)
        cases.append((x, w, torch.randint(0, V, (M,), device=DEV, generator=g), torch.rand(M, device=DEV, generator=g)))

    def step(x, w, labels, dloss, stream=None):
        loss, lse = wb.linear_cross_entropy(x, w, labels, stream=stream)
        return (loss, lse, *wb.linear_cross_entropy_backward(dloss, x, w, labels, lse, stream=stream))

    want = [step(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(5):
        for i, c in enumerate(cases):
            got[i].append(step(*c, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)
    assert wb.check_device_error() == 0


def test_two_graphs_of_the_same_calls_replayed_together(wb):
    M, d, V = 300, 384, 4000
    g = torch.Generator(device=DEV).manual_seed(7)
    w = (torch.randn(V, d, device=DEV, generator=g) * 0.1).to(torch.bfloat16)
    graphs, outs, refs = [], [], []
    for _ in range(2):
        x = torch.randn(M, d, device=DEV, generator=g).to(torch.bfloat16)
        labels = torch.randint(0, V, (M,), device=DEV, generator=g)
        dl = torch.rand(M, device=DEV, generator=g)

        def step():
            loss, lse = wb.linear_cross_entropy(x, w, labels)
            return (loss, lse, *wb.linear_cross_entropy_backward(dl, x, w, labels, lse))

        refs.append(step())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append((graph, x, labels, dl))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(outs[i], refs[i]):
            assert torch.equal(a, b)


FIRST_CALL = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import whisper_encoder_gb300 as wb
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(200, 768, device="cuda", generator=g).bfloat16()
w = (torch.randn(900, 768, device="cuda", generator=g) * 0.1).bfloat16()
lab = torch.randint(0, 900, (200,), device="cuda", generator=g)
ga, be = torch.rand(768, device="cuda"), torch.rand(768, device="cuda")
def step():
    y, total, stats = wb.layernorm_forward(x, ga, be)
    loss, lse = wb.linear_cross_entropy(y, w, lab)
    dx, dw = wb.linear_cross_entropy_backward(torch.ones_like(loss), y, w, lab, lse)
    one = wb.linear_cross_entropy(y[:1], w, lab[:1])
    return (loss, dx, dw, *one, *wb.layernorm_backward(dx, total, ga, stats))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
assert wb.check_device_error() == 0
print("first call captured")
"""


def test_a_first_call_that_is_captured(wb):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first call captured" in r.stdout, r.stderr[-2000:]
