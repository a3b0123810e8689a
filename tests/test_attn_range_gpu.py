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


def large_values(n, heads, D, dt, g):
    """Values of half of bf16's largest: a column of them, one of either sign, one of zeros, one of every other token."""
    big = torch.finfo(torch.bfloat16).max / 2
    v = torch.full((n, heads, D), big, device=DEV)
    v[:, :, 1::4] *= torch.randint(0, 2, (n, heads, (D + 2) // 4), device=DEV, generator=g) * 2.0 - 1.0
    v[:, :, 2::4] = 0.0
    v[::2, :, 3::4] = 0.0
    return v.to(dt)


def written(lengths, heads, D, bits, dt, page=16, seed=0):
    """Sequences of large values as qa_kv_write stores them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    seqs = []
    for n in lengths:
        pages = -(-n // page)
        w, cdt = (D, torch.int8) if bits == 8 else (D // 8, torch.int32)
        mk = lambda *s, t=torch.float32: torch.zeros(pages, heads, page, *s, dtype=t, device=DEV)   # noqa: E731
        cache = (mk(w, t=cdt), mk(), mk(w, t=cdt), mk())
        k = torch.randn(n, heads, D, device=DEV, generator=g).to(dt)
        qa.qa_kv_write(k, large_values(n, heads, D, dt, g), torch.arange(n, device=DEV), cache)
        flat = lambda x: x.transpose(1, 2).flatten(0, 1)[:n]                                         # noqa: E731
        kc, ks, vc, vs = (flat(x) for x in cache)
        kc, vc = (kc.long(), vc.long()) if bits == 8 else (unpack(kc), unpack(vc))
        assert torch.isfinite(vs).all() and float(vs.max()) >= 2.0 ** 118
        seqs.append((kc, ks, vc, vs))
    return seqs, g


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bits", [8, 4])
def test_values_near_the_largest_numbers(bits, dt):
    seqs, g = written([300, 40, 1], 2, 64, bits, dt)
    q = torch.randn(3, 4, 64, device=DEV, generator=g).to(dt)
    got, _ = check(Cached(seqs, bits), q, 0.125, dt)
    assert (got[:, :, 2::4] == 0).all()


@pytest.mark.parametrize("n", [1500, 20000])
@pytest.mark.parametrize("bits", [8, 4])
def test_values_near_the_largest_numbers_in_parts(bits, n):
    seqs, g = written([n], 2, 64, bits, torch.float32, seed=1)
    q = torch.randn(1, 4, 64, device=DEV, generator=g)
    assert qa.qa_attn_decode_workspace(1, 4, 2, 64, n) > 0
    got, _ = check(Cached(seqs, bits), q, 0.125)
    assert (got[:, :, 2::4] == 0).all()


def two_heads(x0, x1, vs, bits=8, seed=2, D=16):
    """One key head under two queries that read a channel each: scores x0 and x1 (whole numbers), value scales vs."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = len(vs)
    kc = torch.zeros(n, 1, D, dtype=torch.int64, device=DEV)
    kc[:, 0, 0], kc[:, 0, 1] = torch.tensor(x0, device=DEV), torch.tensor(x1, device=DEV)
    q = torch.zeros(1, 2, D, device=DEV)
    q[0, 0, 0] = q[0, 1, 1] = 1.0
    return (kc, torch.ones(n, 1, device=DEV), codes(g, n, 1, D, bits=bits), torch.tensor(vs, device=DEV)[:, None]), q


@pytest.mark.parametrize("dt", [torch.float32, torch.float16])
@pytest.mark.parametrize("order", [24, 27, 60, 110])
def test_a_tile_far_below_while_another_head_grows(order, dt):
    """Head 0 sees tokens near its largest, then a tile of each wave without weight, then such tokens again; head 1's
    largest moves in the tile without weight."""
    x0 = [0] * 128 + [-120] * 128 + [-(t % 3) for t in range(128)]
    x1 = [0] * 128 + [40] * 128 + [0] * 128
    s, q = two_heads(x0, x1, [2.0 ** -order] * 384)
    check(Cached([s]), q.to(dt), 1.0, exact_queries=True)


@pytest.mark.parametrize("order", [10, 27, 60, 110])
def test_value_scales_of_zero_before_small_ones(order):
    s, q = two_heads([0] * 256, [1] * 256, [0.0] * 128 + [2.0 ** -order] * 128)
    check(Cached([s]), q, 1.0, exact_queries=True)


def first_far_above(n, nats, bits=8, D=16, seed=3):
    """A first token whose score is `nats` above the equal ones of n - 1 others; its values leave every other channel."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    kc = torch.zeros(n, 1, D, dtype=torch.int64, device=DEV)
    kc[0, 0, 0] = 7
    ks = torch.full((n, 1), nats / 7.0, device=DEV)
    vc = codes(g, n, 1, D, bits=bits).abs()
    vc[0, 0, ::2] = 0
    q = torch.zeros(1, 1, D, device=DEV)
    q[0, 0, 0] = 1.0
    return (kc, ks, vc, torch.rand(n, 1, device=DEV, generator=g) + 0.5), q


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("nats", [10.0, 14.0, 17.5, 20.0])
def test_many_small_weights_beside_one(nats, bits):
    """One block takes the whole sequence, as with many sequences: where the first token's values are 0, the sum of the
    others is the output."""
    s, q = first_far_above(32768, nats, bits)
    short = tuple(x[:1] for x in s)
    c = Cached([s] + [short] * 767, bits)
    c.lengths[1:] = 0
    c.seqs = c.seqs[:1]
    assert qa.qa_attn_decode_workspace(768, 1, 1, 16, 32768) == 0
    q = q.expand(768, 1, 16).contiguous()
    check(c, q, 1.0, exact_queries=True)


@pytest.mark.parametrize("nats", [10.0, 17.5])
def test_many_small_weights_beside_one_in_parts(nats):
    s, q = first_far_above(32768, nats)
    check(Cached([s]), q, 1.0, exact_queries=True)


@pytest.mark.parametrize("step", [0.9, 0.3, 1.7])
def test_references_that_move_by_parts_of_a_binary_order(step):
    """Head 1's scores move its reference in every tile of a wave and head 0's with it, by `step` binary orders;
    the values' scales make up for it, so that head 0's first tokens and its last ones weigh the same."""
    tiles = 60
    i = torch.arange(128 * tiles, device=DEV) // 128
    n = 128 * tiles
    g = torch.Generator(device=DEV).manual_seed(4)
    kc = torch.zeros(n, 1, 16, dtype=torch.int64, device=DEV)
    kc[:, 0, 0] = i
    vs = torch.where(i == 0, 1.0, torch.exp2(-step * (tiles - 1) * torch.ones_like(i, dtype=torch.float32)))
    s = (kc, torch.ones(n, 1, device=DEV), codes(g, n, 1, 16), vs[:, None])
    q = torch.zeros(768, 2, 16, device=DEV)
    q[:, 0, 0], q[:, 1, 0] = 1.0, 64.0
    c = Cached([s] + [tuple(x[:1] for x in s)] * 767)
    c.lengths[1:] = 0
    c.seqs = c.seqs[:1]
    check(c, q, step * math.log(2.0), exact_queries=True)


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


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
def test_scores_that_grow_with_exact_digits(dt, bits):
    """Scores that are whole numbers and grow from tile to tile: the references move again and again, and the values
    are checked to the digits of the sums."""
    n, D = 3000, 64
    g = torch.Generator(device=DEV).manual_seed(8)
    kc = torch.zeros(n, 1, D, dtype=torch.int64, device=DEV)
    kc[:, 0, 1] = torch.arange(n, device=DEV) % 4 + (0 if bits == 4 else torch.arange(n, device=DEV) // 100)
    q = torch.zeros(1, 3, D, device=DEV, dtype=dt)
    q[0, 0, 1], q[0, 1, 1], q[0, 2, 1] = 1.0, -1.0, 16.0
    s = (kc, torch.ones(n, 1, device=DEV), codes(g, n, 1, D, bits=bits), torch.rand(n, 1, device=DEV, generator=g) + 0.5)
    check(Cached([s], bits), q, 1.0, exact_queries=True)


def shared_case(D=64, bits=8, n=5000, seed=9):
    g = torch.Generator(device=DEV).manual_seed(seed)
    most = 127 if bits == 8 else 7
    seqs = [(codes(g, m, 2, D, bits=bits), (torch.rand(m, 2, device=DEV, generator=g) + 0.2) / most,
             codes(g, m, 2, D, bits=bits), (torch.rand(m, 2, device=DEV, generator=g) + 0.2) / most) for m in (n, n // 3, 200)]
    return Cached(seqs, bits), torch.randn(3, 4, D, device=DEV, generator=g)


@pytest.mark.parametrize("where", [1, 3])
@pytest.mark.parametrize("at", [0, 1234, 4999])
def test_nan_scales_through_the_join(at, where):
    c, q = shared_case()
    assert qa.qa_attn_decode_workspace(3, 4, 2, 64, 5008) > 0
    clean, clean_lse = qa.qa_attn_decode(q, c.tensors, c.table, c.lengths, want_lse=True)
    c.tensors[where][int(c.table[0, at // 16]), 1, at % 16] = math.nan
    got, lse = qa.qa_attn_decode(q, c.tensors, c.table, c.lengths, want_lse=True)
    assert torch.isnan(got[0, 2:]).all()
    assert torch.equal(got[0, :2], clean[0, :2]) and torch.equal(got[1:], clean[1:])
    assert torch.isnan(lse[0, 2:]).all() if where == 1 else torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_queries_without_a_finite_value_through_the_join(dt):
    c, q = shared_case()
    q = q.to(dt)
    clean, clean_lse = qa.qa_attn_decode(q, c.tensors, c.table, c.lengths, want_lse=True)
    q[0, 1, 63], q[1, 2, 0], q[1, 3, 5] = math.inf, math.nan, -math.inf
    got, lse = qa.qa_attn_decode(q, c.tensors, c.table, c.lengths, want_lse=True)
    bad = torch.zeros(3, 4, dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[1, 2] = bad[1, 3] = True
    assert torch.isnan(got[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(got[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [176, 208, 256])
def test_large_heads_in_parts(D, bits):
    c, q = shared_case(D, bits, seed=10)
    for dt in (torch.float32, torch.bfloat16):
        check(c, q.to(dt), D ** -0.5, dt)
