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


# Adapters: the last of many against a call that has it alone, and tokens that repeat.
@pytest.mark.parametrize("M,K,N,r,L", [(5, 32768, 64, 256, 280), (100, 32768, 64, 256, 280),       # A past 4 GiB
                                       (5, 16, 12288, 256, 720), (100, 16, 32768, 256, 270)])      # B
def test_last_adapter(M, K, N, r, L):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    n = lambda *s: torch.randn(*s, device=DEV, generator=g)
    A = torch.zeros(L, r, K, dtype=torch.float16, device=DEV)
    B = torch.zeros(L, N, r, dtype=torch.float16, device=DEV)
    assert max(A[:-1].nbytes, B[:-1].nbytes) > 1 << 32
    A[-1], B[-1] = n(r, K).half(), n(N, r).half()
    X, Xq = n(M, K).half(), (n(M, K) * 32).round().clamp(-127, 127).to(torch.int8)
    Wq = (n(N, K) * 32).round().clamp(-127, 127).to(torch.int8)
    s_x, s_w = torch.rand(M, device=DEV, generator=g) / 32, torch.rand(N, device=DEV, generator=g) / 32
    alpha = torch.ones(L, device=DEV)
    seg = torch.tensor([0, M // 2, M], dtype=torch.int32, device=DEV)
    which = torch.tensor([L - 1, -1], dtype=torch.int32, device=DEV)
    got = qa.qa_qlinear_int8_lora(Xq, s_x, X, Wq, s_w, A, B, alpha, seg, which, out_dtype=torch.float32)
    which = torch.tensor([0, -1], dtype=torch.int32, device=DEV)
    want = qa.qa_qlinear_int8_lora(Xq, s_x, X, Wq, s_w, A[-1:].clone(), B[-1:].clone(), alpha[:1], seg, which,
                                   out_dtype=torch.float32)
    none = qa.qa_qlinear_int8_lora(Xq, s_x, X, Wq, s_w, A[-1:], B[-1:], alpha[:1], seg, torch.full_like(which, -1),
                                   out_dtype=torch.float32)
    assert torch.equal(got, want) and not torch.equal(got[:M // 2], none[:M // 2])


def test_parts_of_many_inner_products():
    """540000 tokens, K in 8 parts, 8 groups of ranks: the parts fill 4.4 GB, the tokens' values 8.8."""
    M, n, K, N, r = 540000, 1000, 8192, 48, 256
    g = torch.Generator(device=DEV).manual_seed(7)
    X0 = torch.randn(n, K, device=DEV, generator=g).half()
    Q0 = (torch.randn(n, K, device=DEV, generator=g) * 32).round().clamp(-127, 127).to(torch.int8)
    s0 = torch.rand(n, device=DEV, generator=g) / 32
    Wq = (torch.randn(N, K, device=DEV, generator=g) * 32).round().clamp(-127, 127).to(torch.int8)
    s_w = torch.rand(N, device=DEV, generator=g) / 32
    A, B = torch.randn(1, r, K, device=DEV, generator=g).half(), torch.randn(1, N, r, device=DEV, generator=g).half()
    alpha, which = torch.ones(1, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda Q, s, X, m: qa.qa_qlinear_int8_lora(Q, s, X, Wq, s_w, A, B, alpha,
                                                      torch.tensor([0, m], dtype=torch.int32, device=DEV), which)
    assert qa.qa_qlinear_int8_lora_workspace(M, K, r) > 1 << 32
    want = call(Q0, s0, X0, n)
    got = call(Q0.repeat(M // n, 1), s0.repeat(M // n), X0.repeat(M // n, 1), M).view(M // n, n, N)
    for i in (0, 1, M // n // 2, M // n - 1):
        assert torch.equal(got[i], want), i
