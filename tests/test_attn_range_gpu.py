"""Attention of one token per sequence where its numbers are far apart: the ranges of scales, weights, scores and queries,
against softmax attention in 64 bits on the values that the codes stand for.

Tolerance of an output, before any run: with u = 2^-24, X the largest score's magnitude and n the tokens,
  scores: exact sums of the codes and the queries' whole numbers, 2^-30 (fp32 queries) or 2^-22 of the head's largest
  query times sum |k|; the factors, the sums' two halves and the difference from the reference are 10 roundings of X;
  weights: exp2, p s_v and its two fp16 numbers, 2^-21 of each, and 2^-37 of the largest weight (half a step of the
  smallest fp16 numbers, 2^-25, beside a largest of 2^12 or more) times the codes;
  sums: n / 32 + 64 additions in a row at most, u each, of A = sum_t p_t |v_t|, in the numerator and the denominator;
  and half a step of the output's type."""
import math

import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def pack(q):
    """Codes int64 [..., D] -> int32 words."""
    x = ((q & 15).reshape(*q.shape[:-1], -1, 8) << torch.arange(0, 32, 4, device=q.device)).sum(-1)
    return torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32)


def unpack(w):
    x = (w.long()[..., None] >> torch.arange(0, 32, 4, device=w.device)) & 15
    return torch.where(x > 7, x - 16, x).flatten(-2)


class Cached:
    """Sequences of tokens, each (key codes [n x heads x D], key scales [n x heads], value codes, value scales), in the
    pages of a cache in no order."""

    def __init__(self, seqs, bits=8, page=16, width=None):
        need = [-(-len(s[0]) // page) for s in seqs]
        heads, D = seqs[0][0].shape[1:]
        pages, g = sum(need) + 2, torch.Generator(device=DEV).manual_seed(5)
        order = torch.randperm(pages, device=DEV, generator=g)
        self.table = torch.full((len(seqs), width or max(need)), -1, dtype=torch.int32, device=DEV)
        held = []
        for i in range(4):
            shape = (pages, heads, page) + ((D,) if i % 2 == 0 else ())
            held.append(torch.zeros(shape, dtype=torch.int64 if i % 2 == 0 else torch.float32, device=DEV))
        at = 0
        for b, s in enumerate(seqs):
            mine = order[at:at + need[b]]
            self.table[b, :need[b]] = mine.int()
            at += need[b]
            t = torch.arange(len(s[0]), device=DEV)
            for x, y in zip(held, s):
                x[mine[t // page], :, t % page] = y.to(x.dtype)
        self.seqs = [(s[0].double(), s[1].float().double(), s[2].double(), s[3].float().double()) for s in seqs]
        code = (lambda x: x.to(torch.int8)) if bits == 8 else pack
        self.tensors = (code(held[0]), held[1], code(held[2]), held[3])
        self.lengths = torch.tensor([len(s[0]) for s in seqs], dtype=torch.int32, device=DEV)


def check(c, q, scale, dt=torch.float32, exact_queries=False, **kw):
    """The call's outputs, after a comparison with 64 bits."""
    got, lse = qa.qa_attn_decode(q, c.tensors, c.table, c.lengths, scale=scale, out_dtype=dt, want_lse=True, **kw)
    B, H, D = q.shape
    part = 0.0 if exact_queries else 2.0 ** -30 if q.dtype == torch.float32 else 2.0 ** -22
    for b, (kc, ks, vc, vs) in enumerate(c.seqs):
        n, heads, _ = kc.shape
        for h in range(H):
            g, Q = h // (H // heads), q[b, h].double()
            k, v = kc[:, g] * ks[:, g, None], vc[:, g] * vs[:, g, None]
            x = (k * Q).sum(1) * scale
            p = torch.softmax(x, 0)
            want, A = p @ v, p @ v.abs()
            X = float(x.abs().max())
            off = part * float(Q.abs().max()) * float(k.abs().sum(1).max()) * abs(scale) + 10 * U * X
            least = 2.0 ** -37 * float((p * vs[:, g].abs()).max()) * vc[:, g].abs().sum(0)
            tol = (2 * off + 2 * (n / 32 + 64) * U + 2.0 ** -21) * A + least + torch.finfo(dt).eps / 2 * want.abs()
            err = (got[b, h].double() - want).abs()
            assert (err <= tol).all(), (b, h, float((err / tol.clamp(min=1e-300)).max()))
            assert abs(float(lse[b, h]) - float(torch.logsumexp(x, 0))) <= off + (n / 32 + 64) * U + 4 * U * (X + math.log(n))
    return got, lse


def codes(g, *shape, bits=8):
    most = 127 if bits == 8 else 7
    return torch.randint(-most, most + 1, shape, device=DEV, generator=g)


@pytest.mark.parametrize("n", [400, 5000])
def test_value_scales_below_zero(n):
    """A filled cache may hold them: weights of either sign, larger and larger."""
    g = torch.Generator(device=DEV).manual_seed(6)
    sign = torch.randint(0, 2, (n, 2), device=DEV, generator=g) * 2.0 - 1.0
    for s in (sign, -torch.ones_like(sign)):
        vs = s * torch.exp2(torch.arange(n, device=DEV)[:, None] * (60.0 / n) - 20.0)
        x = (codes(g, n, 2, 64), torch.rand(n, 2, device=DEV, generator=g) / 100, codes(g, n, 2, 64), vs)
        q = torch.randn(1, 4, 64, device=DEV, generator=g)
        check(Cached([x]), q, 0.125)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128, 256, 48])
@pytest.mark.parametrize("large", [1.0, 100.0, 1000.0])
def test_fp32_queries_with_large_channels(large, D, bits):
    """Queries keep their digits beside a few channels far above the others, where the keys may hold zeros."""
    g = torch.Generator(device=DEV).manual_seed(7)
    seqs = []
    for n in (700, 33):
        kc = codes(g, n, 2, D, bits=bits)
        kc[:, :, 3] = kc[:, :, D - 5] = 0
        seqs.append((kc, torch.rand(n, 2, device=DEV, generator=g) * 3 / (127 if bits == 8 else 7),
                     codes(g, n, 2, D, bits=bits), torch.rand(n, 2, device=DEV, generator=g)))
    q = torch.randn(2, 6, D, device=DEV, generator=g)
    q[:, :, 3] *= large
    q[:, :, D - 5] *= large
    check(Cached(seqs, bits), q, D ** -0.5)
