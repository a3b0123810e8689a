"""Norm, routing, experts and adapters give one output, bit for bit, eagerly, on a second stream, and from a captured
graph replayed with other work in between."""
import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def layer(T, K=256, F=96, E=8, k=2, r=16, L=3, N=320):
    """Codes from the norm, the shared projection with adapters, routing and the experts, with all buffers made up front."""
    g = torch.Generator(device=DEV).manual_seed(T)
    n = lambda *s: torch.randn(*s, device=DEV, generator=g)
    codes = lambda *s: (n(*s) * 32).round().clamp(-127, 127).to(torch.int8)
    X, R, w = n(T, K).half(), n(T, K).half(), (n(K).abs() + 0.1).half()
    Wq, s_w = codes(N, K), torch.rand(N, device=DEV, generator=g) / 500
    A, B = (n(L, r, K) / 16).half(), (n(L, N, r) / 4).half()
    alpha = torch.ones(L, device=DEV)
    seg = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device=DEV)
    which = torch.tensor([1, 0, 2], dtype=torch.int32, device=DEV)
    Wr = (n(K, E) / 16).half()
    W13, W2 = codes(E, 2 * F, K), codes(E, K, F)
    s13, s2 = torch.rand(E, 2 * F, device=DEV, generator=g) / 500, torch.rand(E, K, device=DEV, generator=g) / 300
    logits = (X @ Wr).float()

    def call(stream=None):
        q, s, total, y = qa.qa_rmsnorm_int8(X, w, residual=R, want_y=True, stream=stream)
        o = qa.qa_qlinear_int8_lora(q, s, y, Wq, s_w, A, B, alpha, seg, which, stream=stream)
        ids, wt, order, offsets = qa.qa_route_experts(logits, k, stream=stream)
        z = qa.qa_experts_int8(q, s, wt, order, offsets, W13, s13, W2, s2, stream=stream)
        return q, s, total, y, o, ids, wt, order, offsets, z
    return call


@pytest.mark.parametrize("T", [3, 30, 700])
def test_streams_and_graph_replays(T):
    call = layer(T)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        for t in out:
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i
        again = call()                                       # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, again)), i
