"""The cache, the attention and the linear where byte offsets pass 32 bits: what lies at the far end of the arrays gives
what the same data give in small ones."""
import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def cache_of(pages, heads, page, D, bits):
    w, dt = (D, torch.int8) if bits == 8 else (D // 8, torch.int32)
    mk = lambda *s, dt=torch.float32: torch.zeros(pages, heads, page, *s, dtype=dt, device=DEV)     # noqa: E731
    return mk(w, dt=dt), mk(), mk(w, dt=dt), mk()


@pytest.mark.parametrize("bits,pages", [(8, 41000), (4, 82000)])       # 5.4 GB of codes for each of keys and values
def test_far_pages(bits, pages):
    heads, page, D, T, H = 8, 64, 256, 300, 16
    g = torch.Generator(device=DEV).manual_seed(bits)
    k, v = (torch.randn(T, heads, D, device=DEV, generator=g).half() for _ in range(2))
    q = torch.randn(1, H, D, device=DEV, generator=g).half()
    lengths = torch.tensor([T], dtype=torch.int32, device=DEV)
    res = []
    for n, order in ((8, [0, 3, 1, 5, 4]), (pages, [pages - 1, 5, pages // 2 + 7, pages - 2, pages - 40])):
        cache = cache_of(n, heads, page, D, bits)
        table = torch.tensor([order], dtype=torch.int32, device=DEV)
        t = torch.arange(T, device=DEV)
        slots = table[0].long()[t // page] * page + t % page
        qa.qa_kv_write(k, v, slots, cache)
        o, lse = qa.qa_attn_decode(q, cache, table, lengths, want_lse=True)
        res.append((o, lse) + qa.qa_kv_read(slots, cache))
        del cache
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_many_tokens_read_and_written():
    """Inputs and outputs of 4.3 GB: the first tokens over and over."""
    heads, page, D, n, times = 64, 16, 256, 1024, 130
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(n, heads, D, device=DEV, generator=g).half() for _ in range(2))
    small = cache_of(n // page, heads, page, D, 8)
    qa.qa_kv_write(k, v, torch.arange(n, device=DEV), small)
    want = qa.qa_kv_read(torch.arange(n, device=DEV), small)
    kr, vr = qa.qa_kv_read(torch.arange(n, device=DEV).repeat(times), small)
    for got, one in ((kr, want[0]), (vr, want[1])):
        for i in (0, 64, times - 1):
            assert torch.equal(got[i * n:(i + 1) * n], one)
    del kr, vr
    big = cache_of(n * times // page, heads, page, D, 8)
    qa.qa_kv_write(k.repeat(times, 1, 1), v.repeat(times, 1, 1), torch.arange(n * times, device=DEV), big)
    for a, b in zip(big, small):
        for i in (0, 64, times - 1):
            assert torch.equal(a[i * (n // page):(i + 1) * (n // page)], b)


def test_many_queries():
    """Queries and outputs of 4.3 GB in fp32: sequences that share pages."""
    B, H, heads, D, page = 1 << 16, 64, 4, 256, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    cache = cache_of(4, heads, page, D, 8)
    k, v = (torch.randn(64, heads, D, device=DEV, generator=g).half() for _ in range(2))
    qa.qa_kv_write(k, v, torch.arange(64, device=DEV), cache)
    few = torch.randn(16, H, D, device=DEV, generator=g)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    lengths = (torch.arange(16, device=DEV) + 10).int()
    want = qa.qa_attn_decode(few, cache, table.expand(16, 2).contiguous(), lengths, window=64)
    got = qa.qa_attn_decode(few.repeat(B // 16, 1, 1), cache, table.expand(B, 2).contiguous(), lengths.repeat(B // 16), window=64)
    for i in (0, 3000, B // 16 - 1):
        assert torch.equal(got[16 * i:16 * i + 16], want)


def test_linear_rows():
    M, K, N, n = 600064, 64, 4096, 1024                      # 4.9 GB of outputs and of residuals
    g = torch.Generator(device=DEV).manual_seed(3)
    codes = lambda *s: torch.randint(-127, 128, s, device=DEV, generator=g).to(torch.int8)     # noqa: E731
    X, W, s_x, s_w = codes(n, K), codes(N, K), torch.rand(n, device=DEV, generator=g), torch.rand(N, device=DEV, generator=g) / 99
    r = torch.randn(n, N, device=DEV, generator=g).half()
    want = qa.qa_qlinear_int8_act(X, s_x, W, s_w, residual=r)
    res = r.repeat(M // n, 1)
    out = qa.qa_qlinear_int8_act(X.repeat(M // n, 1), s_x.repeat(M // n), W, s_w, residual=res, out=res)
    for i in (0, 500, M // n - 1):
        assert torch.equal(out[i * n:(i + 1) * n], want)


@pytest.mark.parametrize("M", [3, 40])
def test_linear_columns(M):
    """Weights of 4.6 GB; the last columns are the first ones again."""
    K, N, n = 65536, 70000, 7000
    g = torch.Generator(device=DEV).manual_seed(4)
    W = torch.randint(-127, 128, (n, K), device=DEV, generator=g, dtype=torch.int8)
    X, s_x = torch.randint(-127, 128, (M, K), device=DEV, generator=g, dtype=torch.int8), torch.rand(M, device=DEV, generator=g)
    s_w = torch.rand(n, device=DEV, generator=g) / 9999
    want = qa.qa_qlinear_int8_act(X, s_x, W, s_w, out_dtype=torch.float32)
    got = qa.qa_qlinear_int8_act(X, s_x, W.repeat(N // n, 1), s_w.repeat(N // n), out_dtype=torch.float32)
    for i in (0, 4, N // n - 1):
        assert torch.equal(got[:, i * n:(i + 1) * n], want)
