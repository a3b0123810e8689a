"""Attention of one token per sequence over the paged cache, against softmax attention in 64 bits on the values that
the codes stand for.

Tolerance of an output, before any run: with u = 2^-24,
  scores: the sum of D products in fp32 and two factors, off by (D + 6) u of S = max_t scale sum_d |q_d k_d|, and with
  fp32 queries 2^-22 S more (two fp16 numbers); in the exponential as many nats;
  p: that and 4 u for exp2 and its argument's rounding, |x - m| u for the difference;
  p s_v as two fp16 numbers 2^-21; sums: n / 128 + 64 additions in a row at most, u each, of A = sum_t p_t |v_t|;
  numerator and denominator both: twice; and half a step of the output's type."""
import math

import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def pack(q):
    """Codes int64 [..., D] -> int32 words."""
    x = (q & 15).reshape(*q.shape[:-1], -1, 8) << torch.arange(0, 32, 4, device=q.device)
    x = x.sum(-1)
    return torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32)


def make(B, lengths, H, heads, D, page, bits, dt="f16", seed=0, width=None, spread=1.0):
    """Queries, a cache whose unused places hold NaN scales, tables in no order and what the cache stands for in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + B + H + D + page + bits)
    need = [-(-n // page) for n in lengths]
    width = max(1, max(need)) if width is None else width
    pages = sum(need) + 3
    qm = 127 if bits == 8 else 7
    made, values = [], []
    for _ in range(2):
        q = torch.randint(-qm, qm + 1, (pages, heads, page, D), device=DEV, generator=g)
        s = torch.rand(pages, heads, page, device=DEV, generator=g) * 3.0 / qm + 0.2 / qm
        if spread != 1.0:                                    # scales over many binary orders
            s = s * torch.exp2(torch.rand(pages, heads, page, device=DEV, generator=g) * spread - spread)
        made += [q.to(torch.int8) if bits == 8 else pack(q), s]
        values.append(q.double() * s.double()[..., None])
    order = torch.randperm(pages, device=DEV, generator=g)
    table = torch.full((B, width), -7, dtype=torch.int32, device=DEV)
    at = 0
    used = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    for b, (n, k) in enumerate(zip(lengths, need)):
        table[b, :k] = order[at:at + k].int()
        for i in range(k):
            used[order[at + i], :max(0, min(page, n - i * page))] = True
        at += k
    nan = float("nan")
    for s in (made[1], made[3]):
        s.masked_fill_(~used[:, None], nan)                  # places that must not be looked at
    q = (torch.randn(B, (H + 2) * D, device=DEV, generator=g) * 1.5).to(DT[dt])[:, :H * D].view(B, H, D)
    return q, tuple(made), values, table, torch.tensor(lengths, dtype=torch.int32, device=DEV)


def reference(q, values, table, lengths, page, scale, window=0, pages=None):
    """-> out, lse in 64 bits, and per output the weighted sum of |v| and the largest sum of a score's magnitudes."""
    B, H, D = q.shape
    heads = values[0].shape[1]
    pages = values[0].shape[0]
    out = torch.zeros(B, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=DEV)
    A, S, span = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    for b, n in enumerate(lengths.tolist()):
        first = max(0, n - window) if window else 0
        t = torch.arange(first, max(n, first), device=DEV)
        p = table[b].long()[t // page] if t.numel() else t
        live = (p >= 0) & (p < pages)
        t, p = t[live], p[live]
        if not t.numel():
            continue
        k = values[0][p, :, t % page].repeat_interleave(H // heads, 1)      # [n x H x D]
        v = values[1][p, :, t % page].repeat_interleave(H // heads, 1)
        prod = k * q[b].double() * scale
        x = prod.sum(2)
        w = torch.softmax(x, 0)
        out[b] = (w[..., None] * v).sum(0)
        A[b] = (w[..., None] * v.abs()).sum(0)
        lse[b] = torch.logsumexp(x, 0)
        S[b] = prod.abs().sum(2).amax(0)
        span[b] = x.amax(0) - x.amin(0)
    return out, lse, A, S, span


def check(q, cache, values, table, lengths, page, window=0, scale=None, odt=None, **kw):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    got, lse = qa.qa_attn_decode(q, cache, table, lengths, window=window, scale=scale, out_dtype=odt, want_lse=True, **kw)
    want, lse64, A, S, span = reference(q, values, table, lengths, page, scale, window)
    n = int(lengths.max())
    x = (D + 6) * U * S + (2.0 ** -22 * S if q.dtype == torch.float32 else 0.0) + 4 * U + span * U
    sums = (n / 128 + 64) * U
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + (2 * x + 2 * sums + 2.0 ** -21)[..., None] * A \
        if torch.is_tensor(x) else None
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25                               # half a step below fp16's normal numbers
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())
    alive = torch.isfinite(lse64)
    assert torch.equal(torch.isfinite(lse), alive) and (lse[~alive] == -math.inf).all()
    lt = x + sums + 4 * U * (lse64.abs() + 1.0)
    assert ((lse.double() - lse64).abs()[alive] <= lt[alive]).all()
    assert (got[~alive] == 0).all()
    return got, lse


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 128, 144, 192, 256])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_head_sizes_and_types(D, dt, bits):
    lengths = [1, 37, 200, 0, 16, 129]
    x = make(6, lengths, 6, 2, D, 16, bits, dt, seed=1)
    check(*x, 16)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,heads", [(1, 1), (8, 8), (7, 1), (16, 1), (17, 1), (40, 2), (96, 3), (10, 5)])
def test_groups(H, heads, bits):
    x = make(3, [77, 300, 5], H, heads, 64, 16, bits, seed=2)
    check(*x, 16)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("page", [16, 32, 64, 256, 1024])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1000, 1025])
def test_lengths_and_pages(n, page, bits):
    x = make(2, [n, max(0, n - 1)], 4, 2, 128, page, bits, seed=3)
    check(*x, page)
    check(*x, page, max_len=n)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("B,n", [(1, 5000), (1, 40000), (2, 20001), (40, 1500), (300, 700)])
def test_splits(B, n, bits):
    """One long sequence over the whole card, a few, many: parts of all counts, ragged lengths, empty parts."""
    lengths = [n if i == B // 2 else (i * 9176 + 11) % (n + 1) for i in range(B)]
    x = make(B, lengths, 8, 2, 64, 32, bits, "f32", seed=4)
    a = check(*x, 32, max_len=n)
    b = check(*x, 32, max_len=n)                             # the same bits again
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128, 160])
@pytest.mark.parametrize("B,H,heads", [(1, 4, 2), (7, 20, 1), (60, 6, 3), (700, 1, 1), (1024, 2, 1)])
def test_work_shared_over_short_sequences(B, H, heads, D, bits):
    """Tables far wider than the sequences: shares that hold many of them, of all lengths from 0 on, and one that is long."""
    lengths = [(i * 131 + 77) % 260 if i % 5 else 0 for i in range(B)]
    lengths[B // 3] = 1900
    x = make(B, lengths, H, heads, D, 32, bits, "f16", seed=23, width=300)
    a = check(*x, 32)
    b = check(*x, 32)                                        # the same bits again
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x[3][B // 2:, :3] = -1                                   # sequences whose first pages, or all, are gone
    check(*x, 32)
    x[4].zero_()
    got, lse = qa.qa_attn_decode(x[0], x[1], x[3], x[4], want_lse=True)
    assert (got == 0).all() and (lse == -math.inf).all()


def test_graphs_on_one_workspace():
    """Two captured calls of shared work on one workspace, replayed in turn with the lengths going on between."""
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    calls, graphs, outs = [], [], []
    for i, (B, H, heads) in enumerate([(3, 8, 2), (40, 4, 4)]):
        q, cache, values, table, lengths = make(B, [1500] * B, H, heads, 64, 16, 8, seed=24 + i, width=600)
        lengths -= torch.arange(B, dtype=torch.int32, device=DEV) * 30
        calls.append((q, cache, table, lengths))
        assert qa.qa_attn_decode_workspace(B, H, heads, 64, 9600) > 0
        qa.qa_attn_decode(*calls[i], workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(qa.qa_attn_decode(*calls[i], workspace=ws, want_lse=True))
    for turn in range(4):
        for i in (0, 1):
            calls[i][3].sub_(17 * turn)
            ws.fill_(0xff)                                   # (NaNs: nothing in it lasts from call to call)
            graphs[i].replay()
            want = qa.qa_attn_decode(*calls[i], want_lse=True)
            assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])


@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 100, 128, 1000, 4096])
def test_windows(window):
    lengths = [4000, 100, 33, 32, 1, 0, 129, 2047]
    x = make(8, lengths, 8, 4, 64, 16, 8, "f16", seed=5)
    check(*x, 16, window=window)
    check(*x, 16, window=window, max_len=4000)


def test_masked_pages():
    """Pages that the cache does not have mask their tokens; a sequence with none left gives zeros."""
    q, cache, values, table, lengths = make(4, [500, 64, 200, 48], 4, 2, 128, 16, 8, seed=6)
    table[0, :20] = -1                                       # evicted ones before a window
    table[0, 25] = cache[0].shape[0]                         # one past the last
    table[1] = -1
    table[2, 0] = torch.iinfo(torch.int32).max
    table[2, -1] = torch.iinfo(torch.int32).min
    check(q, cache, values, table, lengths, 16)
    got, lse = qa.qa_attn_decode(q, cache, table, lengths, want_lse=True)
    assert (got[1] == 0).all() and (lse[1] == -math.inf).all()


def test_lengths_out_of_range():
    q, cache, values, table, lengths = make(3, [100, 100, 100], 4, 2, 64, 16, 8, seed=7)
    odd = torch.tensor([-5, 1 << 30, 100], dtype=torch.int32, device=DEV)
    got, lse = qa.qa_attn_decode(q, cache, table, odd, max_len=100, want_lse=True)
    want, lse2 = check(q, cache, values, table, torch.tensor([0, 100, 100], dtype=torch.int32, device=DEV), 16, max_len=100)
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    # shorter than the sequences: the first max_len tokens
    check(q, cache, values, table, torch.tensor([0, 40, 40], dtype=torch.int32, device=DEV), 16, max_len=40)


@pytest.mark.parametrize("odt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_output_types(dt, odt):
    x = make(2, [300, 41], 4, 2, 128, 16, 8, dt, seed=8)
    check(*x, 16, odt=DT[odt])


@pytest.mark.parametrize("bits", [8, 4])
def test_scales_over_many_orders(bits):
    """Values (and keys) whose scales run over 2^40: the sum keeps the digits of what carries it."""
    x = make(3, [2000, 300, 31], 8, 2, 64, 16, bits, "f32", seed=9, spread=40.0)
    check(*x, 16)


def test_scores_that_grow_along_the_sequence():
    """The running maximum has to move again and again: keys of ever larger scale, a large score factor."""
    q, cache, values, table, lengths = make(2, [3000, 700], 4, 2, 64, 16, 8, "f32", seed=10)
    for b in range(2):
        for i in range(-(-int(lengths[b]) // 16)):
            p = int(table[b, i])
            f = 1.0 + i * 0.5
            cache[1][p] *= f
            values[0][p] = cache[0][p].double() * cache[1][p].double()[..., None]
    values[0] = torch.nan_to_num(values[0])
    check(q, cache, values, table, lengths, 16, scale=0.5)


def test_one_token_carries_all():
    """A score far above the others, at the first, a middle and the last place: the output is that token's values."""
    for at in (0, 777, 1999):
        q, cache, values, table, lengths = make(1, [2000], 2, 1, 64, 16, 8, "f32", seed=11)
        p, o = int(table[0, at // 16]), at % 16
        cache[0][p, 0, o] = (q[0, 0].sign() * 127).to(torch.int8)
        cache[1][p, 0, o] = 100.0
        values[0][p, 0, o] = cache[0][p, 0, o].double() * 100.0
        got, _ = check(q, cache, values, table, lengths, 16)
        assert torch.allclose(got[0, 0].double(), values[1][p, 0, o], rtol=2.0 ** -20)


@pytest.mark.parametrize("where", [0, 2])
def test_nan_scales_reach_their_head_alone(where):
    q, cache, values, table, lengths = make(2, [300, 300], 4, 2, 64, 16, 8, seed=12)
    clean = qa.qa_attn_decode(q, cache, table, lengths)
    cache[where + 1][int(table[0, 3]), 1, 5] = float("nan")
    got, lse = qa.qa_attn_decode(q, cache, table, lengths, want_lse=True)
    assert torch.isnan(got[0, 2:]).all()
    assert torch.equal(got[0, :2], clean[0, :2]) and torch.equal(got[1], clean[1])
    assert torch.isnan(lse[0, 2:]).all() == (where == 0)


def test_queries_of_extreme_magnitude():
    for dt, f in (("f32", 1e30), ("f32", 1e-30), ("bf16", 1e30), ("f16", 2.0 ** -22)):
        q, cache, values, table, lengths = make(2, [200, 17], 4, 2, 64, 16, 8, dt, seed=13)
        q = (q.double() * f).to(DT[dt])
        check(q, cache, values, table, lengths, 16, scale=0.125 / f)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("bits", [8, 4])
def test_queries_without_a_finite_value_reach_their_row_alone(dt, bits):
    q, cache, values, table, lengths = make(3, [300, 0, 40], 4, 2, 64, 16, bits, dt, seed=21)
    clean, clean_lse = qa.qa_attn_decode(q, cache, table, lengths, want_lse=True)
    q = q.clone()
    q[0, 1, 63] = math.inf
    q[1, 2, 0] = math.nan                                    # (of a sequence without tokens: zeros as before)
    q[2, 3, 17] = math.nan
    q[2, 0, 5] = -math.inf
    got, lse = qa.qa_attn_decode(q, cache, table, lengths, want_lse=True)
    bad = torch.zeros(3, 4, dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[2, 3] = bad[2, 0] = True
    assert torch.isnan(got[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(got[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])


def test_a_cache_without_pages():
    q, cache, values, table, lengths = make(2, [300, 40], 4, 2, 64, 16, 8, seed=22)
    o, lse = qa.qa_attn_decode(q, tuple(t[:0] for t in cache), table, lengths, want_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()


def test_strided_tables_and_outputs():
    q, cache, values, table, lengths = make(3, [100, 250, 9], 4, 2, 128, 16, 8, seed=14)
    wide = torch.full((3, 64), -3, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    out = torch.full((3, 4, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    got = qa.qa_attn_decode(q, cache, wide[:, :table.shape[1]], lengths, out=out)
    assert got is out
    want = reference(q, values, table, lengths, 16, 128 ** -0.5)[0]
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all()
    ws = torch.empty(qa.qa_attn_decode_workspace(3, 4, 2, 128, 250), dtype=torch.uint8, device=DEV)
    again = qa.qa_attn_decode(q, cache, table, lengths, max_len=250, workspace=ws, out_dtype=torch.bfloat16)
    assert ((again.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all()


def test_no_sequences():
    q, cache, values, table, lengths = make(1, [5], 4, 2, 64, 16, 8)
    o, lse = qa.qa_attn_decode(q[:0], cache, table[:0], lengths[:0], want_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o, lse = qa.qa_attn_decode(q, cache, table[:, :0], lengths, want_lse=True)     # no table at all
    assert (o == 0).all() and (lse == -math.inf).all()


def test_written_then_attended():
    """The cache as qa_kv_write fills it, token by token and in a prompt, serves the attention."""
    B, H, heads, D, page = 3, 8, 2, 64, 16
    g = torch.Generator(device=DEV).manual_seed(20)
    for bits in (8, 4):
        w, cdt = (D, torch.int8) if bits == 8 else (D // 8, torch.int32)
        mk = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=DEV)
        cache = (mk(12, heads, page, w, dt=cdt), mk(12, heads, page), mk(12, heads, page, w, dt=cdt), mk(12, heads, page))
        table = torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4).flip(1).contiguous()
        start = torch.tensor([33, 0, 17], device=DEV)
        slots = torch.cat([table[b].long()[torch.arange(n, device=DEV) // page] * page + torch.arange(n, device=DEV) % page
                           for b, n in enumerate(start.tolist())])
        k, v = (torch.randn(50, heads, D, device=DEV, generator=g).half() for _ in range(2))
        qa.qa_kv_write(k, v, slots, cache)
        for step in range(3):
            at = start + step
            new = table.long().gather(1, (at // page)[:, None])[:, 0] * page + at % page
            qkv = torch.randn(B, (H + 2 * heads) * D, device=DEV, generator=g).half()
            q = qkv[:, :H * D].view(B, H, D)
            qa.qa_kv_write(qkv[:, H * D:(H + heads) * D].view(B, heads, D), qkv[:, (H + heads) * D:].view(B, heads, D), new, cache)
            lengths = (at + 1).int()
            every = torch.arange(12 * page, device=DEV)
            kr, vr = qa.qa_kv_read(every, cache, out_dtype=torch.float32)
            values = [t.view(12, page, heads, D).transpose(1, 2).double() for t in (kr, vr)]
            # (the values read back are q s rounded to fp32, 2^-24 off the product: within the scores' part)
            check(q, cache, values, table, lengths, page)


def test_refusals():
    q, cache, values, table, lengths = make(2, [50, 60], 4, 2, 64, 16, 8)
    with pytest.raises(TypeError):
        qa.qa_attn_decode(q.double(), cache, table, lengths)
    with pytest.raises(TypeError):
        qa.qa_attn_decode(q, cache, table.long(), lengths)
    with pytest.raises(TypeError):
        qa.qa_attn_decode(q, cache, table, lengths.long())
    with pytest.raises(ValueError):
        qa.qa_attn_decode(q, cache, table[:1], lengths)
    with pytest.raises(ValueError):
        qa.qa_attn_decode(q, cache, table, lengths[:1])
    with pytest.raises(ValueError):
        qa.qa_attn_decode(q.transpose(0, 1), cache, table, lengths)
    with pytest.raises(ValueError):
        qa.qa_attn_decode(q[:, :, :32], cache, table, lengths)
    with pytest.raises(qa.QAError):                          # 3 query heads of 2 key heads
        qa.qa_attn_decode(q[:, :3], cache, table, lengths)
    with pytest.raises(qa.QAError):
        qa.qa_attn_decode(q, cache, table, lengths, max_len=1 << 20)
    with pytest.raises(qa.QAError):
        qa.qa_attn_decode(q, cache, table, lengths, window=-1)
    with pytest.raises(qa.QAError):
        qa.qa_attn_decode(q, cache, table, lengths, scale=math.inf)
    with pytest.raises(TypeError):
        qa.qa_attn_decode(q, cache, table, lengths, out_dtype=torch.float64)
    with pytest.raises(qa.QAError):                          # a workspace that is too small
        x = make(1, [5000], 4, 2, 64, 16, 8)
        qa.qa_attn_decode(x[0], x[1], x[3], x[4], workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_refused_workspaces():
    q, cache, values, table, lengths = make(2, [900, 700], 4, 2, 64, 16, 8, seed=26, width=100)
    need = qa.qa_attn_decode_workspace(2, 4, 2, 64, 1600)
    assert need > 0
    with pytest.raises(ValueError):                          # as many elements, not as many bytes
        qa.qa_attn_decode(q, cache, table, lengths, workspace=torch.empty(1, dtype=torch.uint8, device=DEV).expand(need))
    with pytest.raises(TypeError):
        qa.qa_attn_decode(q, cache, table, lengths, workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(qa.QAError):
        qa.qa_attn_decode(q, cache, table, lengths, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    with pytest.raises(qa.QAError):                          # aligned to 256 bytes
        qa.qa_attn_decode(q, cache, table, lengths, workspace=torch.empty(need + 64, dtype=torch.uint8, device=DEV)[16:])
    want = qa.qa_attn_decode(q, cache, table, lengths)
    words = torch.empty(need // 4, dtype=torch.float32, device=DEV)
    assert torch.equal(qa.qa_attn_decode(q, cache, table, lengths, workspace=words), want)
