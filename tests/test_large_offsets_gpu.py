"""Norm, routing and experts where byte offsets pass 32 bits: the last rows (or experts) of arrays that are the first
ones over and over give what the first ones give."""
import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,K", [(280000, 8192), (280001, 8185), (70001, 32768)])
def test_norm(rows, K):
    g = torch.Generator(device=DEV).manual_seed(K)
    base = torch.randn(1000, K, device=DEV, generator=g).half()
    X = torch.empty(rows, K, dtype=torch.float16, device=DEV)
    for r in range(0, rows, 1000):
        X[r:r + 1000] = base[:min(1000, rows - r)]
    w = torch.rand(K, device=DEV, generator=g).half()
    want = qa.qa_rmsnorm_int8(base, w, want_y=True)
    q, s, _, y = qa.qa_rmsnorm_int8(X, w, want_y=True)
    for r in (0, 131000, 262000, rows // 1000 * 1000 - 1000):
        if r + 1000 <= rows:
            assert torch.equal(q[r:r + 1000], want[0]) and torch.equal(s[r:r + 1000], want[1])
            assert torch.equal(y[r:r + 1000], want[3])
    tail = rows % 1000
    if tail:
        assert torch.equal(q[-tail:], want[0][:tail]) and torch.equal(s[-tail:], want[1][:tail])


def test_routing():
    E, k, n, times = 512, 2, 4096, 2048                      # 2^23 tokens, 8.6 GB of logits
    base = torch.randn(n, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).half()
    want = qa.qa_route_experts(base, k)
    ids, w, order, offsets = qa.qa_route_experts(base.repeat(times, 1), k)
    assert torch.equal(ids.view(times, n, k)[-1], want[0]) and torch.equal(w.view(times, n, k)[-1], want[1])
    assert torch.equal(offsets, want[3] * times)
    e = 511                                                  # the last expert's pairs: those of every copy in turn
    mine = want[2][want[3][e]:want[3][e + 1]].long()
    copies = torch.arange(times, device=DEV)[:, None] * (n * k) + mine[None]
    assert torch.equal(order[offsets[e]:offsets[e + 1]].long(), copies.reshape(-1))


@pytest.mark.parametrize("T", [3, 600])
def test_experts(T):
    E, K, F = 70, 32768, 1024                                # 4.7 GB of gate and up weights: a large stride to the last
    g = torch.Generator(device=DEV).manual_seed(T)
    codes = lambda *s: (torch.randn(*s, device=DEV, generator=g) * 32).round().clamp(-127, 127).to(torch.int8)
    W13 = torch.zeros(E, 2 * F, K, dtype=torch.int8, device=DEV)
    W2 = torch.zeros(E, K, F, dtype=torch.int8, device=DEV)
    W13[-1], W2[-1] = codes(2 * F, K), codes(K, F)
    s13, s2 = torch.rand(E, 2 * F, device=DEV, generator=g) / 9000, torch.rand(E, K, device=DEV, generator=g) / 1000
    Xq, s_x = codes(T, K), torch.rand(T, device=DEV, generator=g) / 32
    w = torch.ones(T, 1, device=DEV)
    order = torch.arange(T, dtype=torch.int32, device=DEV)
    last = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    last[-1] = T
    got = qa.qa_experts_int8(Xq, s_x, w, order, last, W13, s13, W2, s2, out_dtype=torch.float32)
    one = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    want = qa.qa_experts_int8(Xq, s_x, w, order, one, W13[-1:].clone(), s13[-1:].clone(), W2[-1:].clone(),
                              s2[-1:].clone(), out_dtype=torch.float32)
    assert torch.equal(got, want) and float(want.abs().max()) > 0
