"""qa_rmsnorm_int8 against the formula in 64 bits, at the sizes, strides and rows where it can go wrong."""
import numpy as np
import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a unit in the last place, relative; and absolute, below the normal numbers
ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}
EPS = 1e-6


def reference(X, R, g, eps=EPS):
    h = X.double() + (0 if R is None else R.double())
    y = h * g.double() / (h.pow(2).mean(1, keepdim=True) + eps).sqrt()
    s = y.abs().amax(1) / 127
    s = torch.where(s > 0, s, torch.ones_like(s))
    return h, y, s


def check(out, X, R, g, dt, eps=EPS):
    q, s, total, y = out
    K = X.shape[1]
    h64, y64, s64 = reference(X.cpu(), None if R is None else R.cpu(), g.cpu(), eps)
    # fp32: a lane's chain of at most K / 1024 + 16 fused terms, then 16 additions in the trees, halved by the square
    # root, and about eight further roundings on the way to y and s
    tol = (48 + K / 1024) * 2.0 ** -24
    assert ((s.cpu().double() - s64).abs() <= tol * s64).all()
    # a code is within half a step of y / s, and the two scales differ by tol
    assert ((q.cpu().double() - y64 / s64[:, None]).abs() <= 0.5 + 127 * 2 * tol).all()
    assert (q.cpu().to(torch.int32).abs() <= 127).all()
    if total is not None:
        want = X.float() if R is None else X.float() + R.float()
        assert torch.equal(total, want.to(DT[dt]))
    if y is not None:
        assert ((y.cpu().double() - y64).abs() <= (ULP[dt] * (1 + tol) + tol) * y64.abs() + TINY[dt]).all()


def make(rows, K, dt, seed=0, residual=True):
    g = torch.Generator(device=DEV).manual_seed(seed + 31 * K + rows)
    X = (torch.randn(rows, K, device=DEV, generator=g) * 2).to(DT[dt])
    R = (torch.randn(rows, K, device=DEV, generator=g) * 3).to(DT[dt]) if residual else None
    w = (torch.rand(K, device=DEV, generator=g) + 0.3).to(DT[dt])
    return X, R, w


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,K", [
    (1, 1), (3, 2), (2, 7), (5, 8), (4, 64), (5, 100), (1, 512), (7, 513), (6, 1000), (5, 1024), (3, 1032), (9, 2048),
    (2, 2049), (1, 4096), (130, 4096), (3, 5001), (4, 8192), (2, 8200), (2, 16384), (2, 16385), (3, 20000)])
def test_against_64_bits(dt, residual, rows, K):
    X, R, w = make(rows, K, dt, residual=residual)
    check(qa.qa_rmsnorm_int8(X, w, residual=R, want_y=True), X, R, w, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K,ld,shift", [(256, 264, 0), (256, 257, 0), (256, 256, 1), (4096, 8200, 3), (96, 200, 8),
                                        (16400, 16410, 1)])
def test_strided_rows_and_odd_starts(dt, K, ld, shift):
    X, R, w = make(5, ld, dt)
    buf = torch.zeros(5 * ld + 16, dtype=DT[dt], device=DEV)
    xv = buf[shift:shift + 5 * ld].view(5, ld)
    xv.copy_(X)
    Xs, Rs, wv = xv[:, :K], R[:, ld - K:], w[:K].clone()
    total = torch.full((5, ld), 7.0, dtype=DT[dt], device=DEV)
    out = qa.qa_rmsnorm_int8(Xs, wv, residual=Rs, want_y=True, total=total[:, :K])
    check((out[0], out[1], total[:, :K], out[3]), Xs, Rs, wv, dt)
    assert (total[:, K:] == 7.0).all()                        # nothing past a row is written


@pytest.mark.parametrize("K", [256, 1001, 4096, 16385])
@pytest.mark.parametrize("into", ["X", "residual"])
def test_sum_in_place(K, into):
    X, R, w = make(6, K, "f16")
    want = qa.qa_rmsnorm_int8(X, w, residual=R, want_y=True)
    x2, r2 = X.clone(), R.clone()
    got = qa.qa_rmsnorm_int8(x2, w, residual=r2, want_y=True, total=x2 if into == "X" else r2)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [512, 4096, 1001, 16400])
def test_rows_without_a_finite_norm(dt, K):
    X, _, w = make(6, K, dt, residual=False)
    clean = qa.qa_rmsnorm_int8(X, w)
    X[1, K // 2] = float("nan")
    X[3, 0] = float("inf")
    X[4] = 0.0
    q, s, _, _ = qa.qa_rmsnorm_int8(X, w)
    assert torch.isnan(s[[1, 3]]).all() and (q[[1, 3]] == 0).all()
    assert s[4] == 1.0 and (q[4] == 0).all()                  # a row of zeros
    for r in (0, 2, 5):
        assert s[r] == clean[1][r] and torch.equal(q[r], clean[0][r])


def test_values_at_the_ends_of_fp32():
    K = 256
    X = torch.randn(4, K, device=DEV)
    w = torch.ones(K, device=DEV)
    X[1] *= 1e30                                              # squares pass fp32
    X[2] *= 1e-25                                             # squares vanish: y = h / sqrt(eps)
    q, s, _, _ = qa.qa_rmsnorm_int8(X, w)
    assert torch.isnan(s[1]) and (q[1] == 0).all()
    _, y64, s64 = reference(X.cpu(), None, w.cpu())
    for r in (0, 2, 3):
        assert abs(float(s[r]) - float(s64[r])) <= 1e-5 * float(s64[r])
        assert ((q[r].cpu().double() - y64[r] / s64[r]).abs() <= 0.51).all()
    tiny = torch.full((K,), 1e-37, device=DEV)                # scales below the normal numbers
    q, s, _, _ = qa.qa_rmsnorm_int8(X[:1], tiny)
    assert float(s[0]) > 0 and int(q.abs().max()) == 127


def test_no_rows():
    q, s, t, y = qa.qa_rmsnorm_int8(torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV), want_y=True)
    assert q.shape == (0, 64) and s.shape == (0,) and y.shape == (0, 64)


def test_codes_feed_the_int8_linear():
    """The codes and scales are those of the row quantizer on the same values, up to the norm's rounding to fp16."""
    X, R, w = make(40, 1024, "f16")
    q, s, _, y = qa.qa_rmsnorm_int8(X, w, residual=R, want_y=True)
    q2, s2 = qa.qa_quantize_rowwise_int8(y)
    assert (q.int() - q2.int()).abs().max() <= 1
    assert ((s - s2).abs() <= 2.0 ** -10 * s).all()


def test_refusals():
    X, R, w = make(4, 64, "f16")
    with pytest.raises(TypeError):
        qa.qa_rmsnorm_int8(X.double(), w.double())
    with pytest.raises(TypeError):
        qa.qa_rmsnorm_int8(X, w.float())
    with pytest.raises(TypeError):
        qa.qa_rmsnorm_int8(X, w, residual=R.float())
    with pytest.raises(ValueError):
        qa.qa_rmsnorm_int8(X, w[:32].clone())
    with pytest.raises(ValueError):
        qa.qa_rmsnorm_int8(X, w, residual=R[:2])
    with pytest.raises(ValueError):
        qa.qa_rmsnorm_int8(X.t(), w[:4].clone())
    with pytest.raises(qa.QAError):
        qa.qa_rmsnorm_int8(X, w, eps=0.0)
