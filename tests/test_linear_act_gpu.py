"""The int8 linear with bias, activation and residual against the formula in 64 bits.

Tolerance, before any run, with u = 2^-24: y = s_x s_w C takes three roundings, + bias one, so x is off by
4 u (|y| + |b|) at most; the activations' slopes are at most 1.2; gelu's own error is 2^-21 of |x| (its polynomial
3e-7, the exponential and four products), silu's and the tanh form's 2^-21 of the result plus what their argument's
four roundings change, 8 u |x| |argument| of a result; the residual's addition one u of the sum; and half a step of the
output's type."""
import math

import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = {"none": qa.QA_ACT_NONE, "relu": qa.QA_ACT_RELU, "gelu": qa.QA_ACT_GELU, "gelu_tanh": qa.QA_ACT_GELU_TANH,
        "silu": qa.QA_ACT_SILU}
U = 2.0 ** -24


def make(M, K, N, seed=0, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed * 131 + M + K + N)
    codes = lambda *s: torch.randint(-127, 128, s, device=DEV, generator=g).to(torch.int8)
    u = lambda *s: torch.rand(*s, device=DEV, generator=g) + 0.5
    return codes(M, K), u(M) / 64, codes(N, K), u(N) * (size * K ** -0.5 / 84), torch.randn(N, device=DEV, generator=g)


def act64(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "gelu":
        return 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
    if act == "gelu_tanh":
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x * torch.sigmoid(x) if act == "silu" else x


def check(got, Xq, s_x, Wq, s_w, bias, act, res):
    y = (Xq.double() @ Wq.double().t()) * s_x.double()[:, None] * s_w.double()
    b = bias.double() if bias is not None else torch.zeros((), dtype=torch.float64, device=DEV)
    x = y + b
    f = act64(x, act)
    want = f + (res.double() if res is not None else 0.0)
    tol = 1.2 * 4 * U * (y.abs() + b.abs()) + torch.finfo(got.dtype).eps / 2 * want.abs() + U * (f.abs() + want.abs())
    if act == "gelu":
        tol = tol + 2.0 ** -21 * x.abs()
    if act in ("silu", "gelu_tanh"):
        arg = x.abs() if act == "silu" else 1.6 * (x.abs() + 0.045 * x.abs() ** 3)
        tol = tol + f.abs() * (2.0 ** -21 + 8 * U * arg.clamp(max=120.0))
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), float((err / tol).max())


# (the last ones: the weight stream's form, ragged columns, K in several parts and ending inside one)
SHAPES = [(1, 16, 1), (1, 64, 16), (3, 80, 17), (16, 256, 100), (17, 128, 33), (32, 512, 48), (33, 144, 130),
          (64, 1040, 64), (65, 96, 200), (130, 272, 131), (200, 512, 1000), (1, 4096, 13000), (16, 4112, 4100),
          (7, 9008, 4113), (16, 80, 8190)]


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_shapes(M, K, N, dt, act):
    x = make(M, K, N)
    res = torch.randn(M, N, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(DT[dt])
    got = qa.qa_qlinear_int8_act(*x[:4], bias=x[4], act=ACTS[act], residual=res)
    assert got.dtype == DT[dt]
    check(got, *x, act, res)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N", [(5, 40), (100, 210)])
def test_without_bias_or_residual(M, N, bias, residual):
    x = make(M, 192, N, seed=1)
    res = torch.randn(M, N, device=DEV) if residual else None
    got = qa.qa_qlinear_int8_act(*x[:4], bias=x[4] if bias else None, act=qa.QA_ACT_SILU, residual=res,
                                 out_dtype=torch.float32)
    check(got, *x[:4], x[4] if bias else None, "silu", res)


# every tile of the product: by the number of tiles (the last one: 128 x 192)
@pytest.mark.parametrize("M,N", [(300, 700), (700, 4096), (1000, 4100), (1030, 8200), (2048, 11008)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_tiles(M, N, act):
    x = make(M, 256, N, seed=2)
    res = torch.randn(M, N, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).bfloat16()
    got = qa.qa_qlinear_int8_act(*x[:4], bias=x[4], act=ACTS[act], residual=res)
    check(got, *x, act, res)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_activations_over_their_range(act):
    """Results from -110 to 110 and dense about zero, in fp32: both tails and the middle."""
    K, N = 16, 4001
    Xq = torch.zeros(1, K, dtype=torch.int8, device=DEV)
    Wq = torch.zeros(N, K, dtype=torch.int8, device=DEV)
    one = torch.ones(1, device=DEV)
    t = torch.linspace(-1.0, 1.0, N, device=DEV)
    for bias in (110.0 * t, 12.0 * t, t ** 5):
        got = qa.qa_qlinear_int8_act(Xq, one, Wq, torch.ones(N, device=DEV), bias=bias, act=ACTS[act], out_dtype=torch.float32)
        want = act64(bias.double(), act)
        # relative where the result is not cancelled: the negative tails too, down to fp32's smallest normal numbers
        arg = (bias.double().abs() if act == "silu" else bias.double() ** 2) if act in ("gelu", "silu") else \
            1.6 * (bias.double().abs() + 0.045 * bias.double().abs() ** 3)
        tol = want.abs() * (2.0 ** -20 + 8 * U * arg.clamp(max=200.0)) + 2.0 ** -126
        if act == "relu":
            tol = torch.zeros_like(tol)
        assert ((got[0].double() - want).abs() <= tol).all()


def test_residual_in_place_and_strided():
    M, K, N = 50, 128, 120
    for M in (10, 50, 300):
        x = make(M, K, N, seed=4)
        wide = torch.randn(M, 3 * N, device=DEV).half()
        before = wide.clone()
        res = before[:, N:2 * N]
        out = wide[:, N:2 * N]
        got = qa.qa_qlinear_int8_act(*x[:4], bias=x[4], residual=out, out=out)
        assert got is out
        check(out, *x, "none", res)
        assert torch.equal(wide[:, :N], before[:, :N]) and torch.equal(wide[:, 2 * N:], before[:, 2 * N:])
        # rows of odd strides and starts: no vector access fits
        odd = torch.zeros(M, N + 3, device=DEV).half()
        got = qa.qa_qlinear_int8_act(*x[:4], residual=before[:, 1:N + 1], out=odd[:, 1:N + 1])
        check(got, *x[:4], None, "none", before[:, 1:N + 1])
        assert (odd[:, 0] == 0).all() and (odd[:, N + 1:] == 0).all()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M", [4, 100])
def test_rows_without_a_finite_scale(M, act):
    x = make(M, 64, 50, seed=5)
    clean = qa.qa_qlinear_int8_act(*x[:4], bias=x[4], act=ACTS[act])
    x[1][2] = float("nan")                                   # as the norm leaves a row that holds an infinity
    got = qa.qa_qlinear_int8_act(*x[:4], bias=x[4], act=ACTS[act])
    assert torch.isnan(got[2]).all()
    rest = [r for r in range(M) if r != 2]
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M,N", [(1, 100), (3, 5000), (100, 70)])
def test_results_past_the_largest_number(M, N, act):
    """Scales whose products pass fp32's largest number: +infinity stays one through every activation."""
    x = make(M, 64, N, seed=6)
    x[0].abs_()
    x[2].abs_()
    x[1].fill_(3e38)
    x[3][::3] = 3e38
    got = qa.qa_qlinear_int8_act(*x[:4], act=ACTS[act], out_dtype=torch.float32)
    assert (got[:, ::3] == math.inf).all() and not torch.isnan(got).any()


def test_the_integer_sum_is_exact():
    """K at the boundary's largest with codes of 127: sums of 2^31 and no rounding before the scales."""
    K, N = 131072, 40
    for M in (2, 70):
        Xq = torch.full((M, K), 127, dtype=torch.int8, device=DEV)
        Wq = torch.full((N, K), -127, dtype=torch.int8, device=DEV)
        one = lambda n: torch.ones(n, device=DEV)
        got = qa.qa_qlinear_int8_act(Xq, one(M), Wq, one(N), out_dtype=torch.float32)
        assert (got == -float(127 * 127 * K)).all()


def test_projection_of_the_mixed_linear():
    """With no outliers, bias, activation or residual it is the LLM.int8() linear on the same codes."""
    g = torch.Generator(device=DEV).manual_seed(6)
    X = torch.randn(24, 512, device=DEV, generator=g).half()
    W = torch.randn(80, 512, device=DEV, generator=g).half()
    Wq, s_w = qa.qa_quantize_rowwise_int8(W)
    Xq, s_x = qa.qa_quantize_rowwise_int8(X)
    a = qa.qa_qlinear_int8_mixed(X, Wq, s_w, threshold=math.inf, out_dtype=torch.float32)
    b = qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, out_dtype=torch.float32)
    assert ((a - b).abs() <= 2.0 ** -22 * a.abs()).all()


def test_no_rows_or_columns():
    x = make(4, 64, 48)
    assert qa.qa_qlinear_int8_act(x[0][:0], x[1][:0], x[2], x[3]).shape == (0, 48)
    assert qa.qa_qlinear_int8_act(x[0], x[1], x[2][:0], x[3][:0]).shape == (4, 0)


def test_refusals():
    Xq, s_x, Wq, s_w, b = make(4, 64, 48)
    res = torch.zeros(4, 48, device=DEV).half()
    with pytest.raises(TypeError):
        qa.qa_qlinear_int8_act(Xq.float(), s_x, Wq, s_w)
    with pytest.raises(ValueError):
        qa.qa_qlinear_int8_act(Xq, s_x[:2], Wq, s_w)
    with pytest.raises(ValueError):
        qa.qa_qlinear_int8_act(Xq, s_x, Wq[:, :32].contiguous(), s_w)
    with pytest.raises(ValueError):
        qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, bias=b[:7])
    with pytest.raises(TypeError):
        qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, bias=b.half())
    with pytest.raises(TypeError):
        qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, residual=res, out=res.float())
    with pytest.raises(ValueError):
        qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, residual=res[:3])
    with pytest.raises(ValueError):
        qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, out=torch.zeros(48, 4, device=DEV).t())
    with pytest.raises(qa.QAError):
        qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, act=9)
    with pytest.raises(TypeError):
        qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, out=torch.zeros(4, 48, device=DEV).double())
