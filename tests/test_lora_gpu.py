"""qa_qlinear_int8_lora against its definition in 64 bits."""
import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def make(M, K, N, r, L, cuts, which, dt="f16", seed=0, x_std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed + M * 5 + K + N * 3 + r)
    n = lambda *s: torch.randn(*s, device=DEV, generator=g)
    X = (n(M, K) * x_std).to(DT[dt])
    s_x = X.float().abs().amax(1) / 127 if M else torch.empty(0, device=DEV)
    Xq = (X.float() / s_x[:, None]).round().to(torch.int8)
    return dict(Xq=Xq, s_x=s_x, X=X, Wq=(n(N, K) * 32).round().clamp(-127, 127).to(torch.int8),
                s_w=(torch.rand(N, device=DEV, generator=g) + 0.5) * (1 / 32 / K ** 0.5),
                A=(n(L, r, K) * K ** -0.5).to(DT[dt]), B=(n(L, N, r) * r ** -0.5).to(DT[dt]),
                alpha=torch.rand(L, device=DEV, generator=g) + 0.5, seg=torch.tensor(cuts, dtype=torch.int32, device=DEV),
                which=torch.tensor(which, dtype=torch.int32, device=DEV))


def check(c, out="f16", dt="f16", **kw):
    got = qa.qa_qlinear_int8_lora(**c, out_dtype=DT[out], **kw)
    D = torch.float64
    p = {n: t.cpu().to(D) for n, t in c.items() if n not in ("seg", "which")}
    M, K = p["Xq"].shape
    base = (p["Xq"] @ p["Wq"].T) * p["s_x"][:, None] * p["s_w"]
    want, room = base.clone(), base.abs() * 4 * 2.0 ** -24
    cuts, which = c["seg"].tolist(), c["which"].tolist()
    # the first product in fp32: K terms, each lane's chain and the trees (at most K / 32 + 16 roundings of the whole,
    # and the products' sums inside a matrix instruction); h as two 16-bit numbers keeps 2^-20 of the row's largest
    # (fp16) or 2^-15 (bf16); the second product: r terms in fp32
    split = 2.0 ** -20 if dt == "f16" else 2.0 ** -15
    for i, a in enumerate(which):
        t = slice(max(0, cuts[i]), min(M, cuts[i + 1]))
        if not 0 <= a < p["A"].shape[0] or t.stop <= t.start:
            continue
        h = p["X"][t] @ p["A"][a].T
        mag = p["X"][t].abs() @ p["A"][a].abs().T
        eh = mag * (K / 32 + 48) * 2.0 ** -24 + h.abs().amax(1, keepdim=True) * split
        Bt = p["B"][a].T
        want[t] += p["alpha"][a] * (h @ Bt)
        room[t] += p["alpha"][a] * (eh @ Bt.abs() + (h.abs() @ Bt.abs()) * (h.shape[1] + 8) * 2.0 ** -24)
    room += want.abs() * 4 * 2.0 ** -24
    g = got.cpu().to(D)
    assert g.shape == want.shape and torch.isfinite(g).all()
    assert ((g - want).abs() <= room + ULP[out] * (want.abs() + room) + TINY[out]).all()
    return got


def spread(M, R, L):
    """Requests of all lengths, empty ones among them, and one without an adapter."""
    cuts = [0] + sorted((i * i * M) // (R * R) for i in range(1, R + 1))
    cuts[-1] = M
    which = [(i * 5 + 1) % L for i in range(R)]
    if R > 2:
        which[R // 2] = -1
    return cuts, which


@pytest.mark.parametrize("dt,out", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("M,K,N,r,L,R", [
    (1, 16, 16, 8, 1, 1), (1, 4096, 48, 16, 2, 1), (2, 80, 33, 8, 3, 2), (16, 256, 100, 16, 4, 16), (17, 528, 65, 24, 5, 9),
    (33, 272, 7, 64, 2, 5), (64, 1024, 130, 128, 3, 20),                                       # few tokens
    (65, 256, 100, 16, 2, 3), (130, 272, 257, 8, 7, 40), (200, 80, 64, 256, 2, 2), (300, 512, 333, 72, 4, 11),
    (777, 128, 640, 32, 8, 48), (1100, 96, 5200, 40, 3, 3)])                                   # tiles, of both sizes
def test_against_64_bits(dt, out, M, K, N, r, L, R):
    check(make(M, K, N, r, L, *spread(M, R, L), dt=dt), out=out, dt=dt)


@pytest.mark.parametrize("M,N", [(1, 12288), (16, 12292), (1, 12289), (32, 8192), (17, 8200), (33, 4096), (64, 4104), (48, 4097)])
def test_both_sides_of_few(M, N):
    check(make(M, 48, N, 24, 3, *spread(M, 4, 3)))


@pytest.mark.parametrize("M,N", [(500, 4096), (513, 3600), (520, 4200), (1030, 4500), (1100, 7700), (129, 16400)])
def test_every_size_of_tile(M, N):
    """K of one whole and one ragged stage."""
    check(make(M, 144, N, 40, 3, *spread(M, 5, 3)), out="f32")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("K", [1040, 2064, 4112, 8208, 9216])
@pytest.mark.parametrize("M,N,r", [(5, 80, 24), (20, 48, 128), (50, 33, 16), (100, 130, 72)])
def test_long_rows(M, N, r, K, dt):
    """K past one batch of the loads of every form, whole and ragged; for many tokens the inner products in 2 to 8 parts."""
    check(make(M, K, N, r, 3, *spread(M, 6, 3), dt=dt), out="f32", dt=dt)


@pytest.mark.parametrize("M", [9, 90])
def test_tokens_outside_every_request(M):
    """The first request starts after token 0 and the last one ends before the end."""
    c = make(M, 64, 40, 16, 2, [3, 3, 6, 6], [0, 1, 0])
    out = check(c)
    none = check({**c, "which": torch.full((3,), -1, dtype=torch.int32, device=DEV)})
    t = torch.ones(M, dtype=torch.bool, device=DEV)
    t[3:6] = False
    assert torch.equal(out[t], none[t]) and not torch.equal(out[3:6], none[3:6])


@pytest.mark.parametrize("M", [5, 80])
def test_requests_past_the_tokens(M):
    check(make(M, 64, 40, 16, 2, [0, M // 2, M + 50], [1, 0]))


@pytest.mark.parametrize("M", [16, 100])
def test_adapters_out_of_range_count_as_none(M):
    c = make(M, 64, 48, 8, 2, [0, M // 2, M], [2, -5])
    plain = qa.qa_qlinear_int8_lora(**{**c, "which": torch.full((2,), -1, dtype=torch.int32, device=DEV)})
    assert torch.equal(check(c), plain)


@pytest.mark.parametrize("M", [6, 70])
def test_no_requests(M):
    c = make(M, 64, 48, 8, 2, [0], [])
    check(c)


@pytest.mark.parametrize("L,R", [(0, 0), (0, 3), (2, 0)])
@pytest.mark.parametrize("M,N", [(4, 48), (20, 48), (64, 48), (100, 48), (700, 4100)])
def test_adapter_arrays_that_are_null(M, N, L, R):
    """Without requests or without adapters X, A, B, alpha, seg and which are not read, in any form of the call."""
    c = make(M, 272, N, 16, 2, [0, M], [-1])
    want = qa.qa_qlinear_int8_lora(**c, out_dtype=torch.float32)
    out = torch.empty(M, N, device=DEV)
    ws = torch.empty(qa.qa_qlinear_int8_lora_workspace(M, 272, 16), dtype=torch.uint8, device=DEV)
    p = lambda t: t.data_ptr()
    s = qa.lib().qa_qlinear_int8_lora(p(c["Xq"]), p(c["s_x"]), None, qa.QA_F16, M, 272, p(c["Wq"]), p(c["s_w"]), N, None,
                                      None, None, 16, L, None, None, R, p(out), qa.QA_F32, p(ws), ws.numel(),
                                      torch.cuda.current_stream().cuda_stream)
    assert s == 0 and qa.last_error() == ""
    assert torch.equal(out, want)


@pytest.mark.parametrize("M", [4, 100])
def test_base_alone_is_the_int8_linear(M):
    c = make(M, 256, 64, 8, 1, [0, M], [-1])
    out = qa.qa_qlinear_int8_lora(**c, out_dtype=torch.float32)
    acc = qa.qa_gemm_i8_i32(c["Xq"], c["Wq"]).double()
    want = acc * c["s_x"].double()[:, None] * c["s_w"].double()
    assert ((out.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("M", [20, 100])
def test_inner_products_past_the_range_of_fp16(M):
    """h up to 1e6 and, in other rows, below fp16's smallest normal number."""
    c = make(M, 512, 64, 16, 2, [0, M // 2, M], [0, 1], x_std=1.0)
    scale = torch.ones(M, 1, device=DEV)
    scale[::2], scale[1::2] = 400.0, 2.0 ** -12
    c["X"] = (c["X"].float() * scale).half()
    c["A"] = (c["A"].float() * 400).half()
    c["B"] = (c["B"].float() * 2.0 ** -10).half()
    check(c, out="f32")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N,top", [(20, 256, 40, 255), (100, 256, 40, 255), (100, 2304, 40, 80), (520, 256, 4200, 255),
                                       (1030, 80, 4520, 255), (1100, 80, 7720, 255)])
def test_inner_products_keep_their_digits(M, K, N, top, dt):
    """Whole numbers below 2^24 with fp32 outputs: every product and sum is exact in fp32, in any order, and each column
    of B picks one rank, so that the outputs are the inner products themselves."""
    g = torch.Generator(device=DEV).manual_seed(M + K)
    n = lambda *s: torch.randint(-top, top + 1, s, device=DEV, generator=g)
    X, A, r = n(M, K), n(2, 40, K), 40
    at = (torch.arange(M, device=DEV) < M // 3).long()
    c = dict(Xq=torch.zeros(M, K, dtype=torch.int8, device=DEV), s_x=torch.ones(M, device=DEV), X=X.to(DT[dt]),
             Wq=torch.zeros(N, K, dtype=torch.int8, device=DEV), s_w=torch.ones(N, device=DEV), A=A.to(DT[dt]),
             B=torch.eye(r, device=DEV).repeat(2, N // r, 1).to(DT[dt]), alpha=torch.ones(2, device=DEV),
             seg=torch.tensor([0, M // 3, M], dtype=torch.int32, device=DEV),
             which=torch.tensor([1, 0], dtype=torch.int32, device=DEV))
    want = torch.stack([X.double() @ A[i].double().T for i in range(2)])[at, torch.arange(M, device=DEV)]
    assert 2 ** 17 < float(want.abs().max()) < 2 ** 22       # past two numbers of bf16, within two of fp16
    out = qa.qa_qlinear_int8_lora(**c, out_dtype=torch.float32)
    assert torch.equal(out.double(), want.repeat(1, N // r))


@pytest.mark.parametrize("M,K,N,r,L,R", [(9, 528, 100, 24, 3, 4), (100, 272, 130, 72, 4, 11), (520, 96, 4200, 40, 3, 5),
                                         (1100, 96, 7700, 16, 3, 6)])
def test_bf16_adapters_with_fp32_outputs(M, K, N, r, L, R):
    check(make(M, K, N, r, L, *spread(M, R, L), dt="bf16"), out="f32", dt="bf16")


@pytest.mark.parametrize("M", [30, 100])
def test_a_broken_adapter_stays_in_its_request(M):
    c = make(M, 128, 64, 16, 2, [0, 10, M], [0, 1])
    clean = qa.qa_qlinear_int8_lora(**c)
    c["B"][1] = float("inf")
    c["A"][1, 3] = float("nan")
    out = qa.qa_qlinear_int8_lora(**c)
    assert torch.equal(out[:10], clean[:10]) and not torch.isfinite(out[10:]).any()


def test_the_same_twice():
    c = make(777, 256, 512, 64, 8, *spread(777, 48, 8))
    assert torch.equal(qa.qa_qlinear_int8_lora(**c), qa.qa_qlinear_int8_lora(**c))


def test_no_tokens():
    c = make(0, 64, 48, 8, 1, [0, 0], [0])
    assert qa.qa_qlinear_int8_lora(**c).shape == (0, 48)


def test_refusals():
    c = make(4, 64, 48, 8, 2, [0, 2, 4], [0, 1])
    for name in ("s_x", "s_w", "alpha", "seg"):
        with pytest.raises(ValueError):
            qa.qa_qlinear_int8_lora(**{**c, name: c[name][:-1].contiguous()})
    with pytest.raises(ValueError):
        qa.qa_qlinear_int8_lora(**{**c, "B": c["B"][:, :40].contiguous()})
    with pytest.raises(TypeError):
        qa.qa_qlinear_int8_lora(**{**c, "X": c["X"].float()})
    with pytest.raises(TypeError):
        qa.qa_qlinear_int8_lora(**{**c, "A": c["A"].bfloat16()})
    with pytest.raises(qa.QAError):
        qa.qa_qlinear_int8_lora(**{**c, "A": c["A"][:, :4].contiguous(), "B": c["B"][:, :, :4].contiguous()})   # r % 8
    with pytest.raises(qa.QAError):
        qa.qa_qlinear_int8_lora(**c, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
