"""The paged cache of int8 and int4 codes: what qa_kv_write stores and qa_kv_read gives back, against the formula in
IEEE fp32 on the host.  Codes, scales and values are defined by single correctly rounded fp32 operations, so they are
compared bit for bit."""
import numpy as np
import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def new_cache(pages, heads, page, D, bits, fill=None):
    """Codes and scales with a pattern that a stray write would change."""
    w, dt = (D, torch.int8) if bits == 8 else (D // 8, torch.int32)
    g = torch.Generator(device=DEV).manual_seed(77)
    codes = lambda: torch.randint(-100, 100, (pages, heads, page, w), device=DEV, generator=g).to(dt)
    scales = lambda: torch.rand(pages, heads, page, device=DEV, generator=g)
    return codes(), scales(), codes(), scales()


def quantize(x, qmax):
    """x fp32 [T x heads x D] on the host -> (codes int64, scales fp32)."""
    x = x.astype(np.float32)
    with np.errstate(invalid="ignore"):
        top = np.abs(x).max(-1)
        bad = ~np.isfinite(x).all(-1)
        s = top / np.float32(qmax)
        s[top == 0] = 1.0
        s[s == 0] = 1.0
        q = np.clip(np.rint(x / s[..., None]), -qmax, qmax)
    s[bad] = np.nan
    q[bad] = 0
    return q.astype(np.int64), s


def unpack(words):
    w = words.cpu().numpy().astype(np.int64)
    q = (w[..., None] >> np.arange(0, 32, 4)) & 15
    return np.where(q > 7, q - 16, q).reshape(*w.shape[:-1], -1)


def rows(t, slots, page):
    return t[slots // page, :, slots % page]


def inputs(T, heads, D, dt, seed, strided=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(T, 3 * heads * D, device=DEV, generator=g) * 2.0).to(DT[dt])
    n = heads * D
    k, v = x[:, n:2 * n].view(T, heads, D), x[:, 2 * n:].view(T, heads, D)
    return (k, v) if strided else (k.clone(), v.clone())


def check(cache, k, v, slots, page, bits):
    """Every place: the new tokens' rows by the formula, all others as they were before."""
    qmax = 127 if bits == 8 else 7
    live = slots >= 0
    for x, codes, scales in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        q, s = quantize(x.float().cpu().numpy()[live.cpu().numpy()], qmax)
        at = slots[live]
        got = rows(codes, at, page)
        got = got.cpu().numpy().astype(np.int64) if bits == 8 else unpack(got)
        assert np.array_equal(got, q)
        assert np.array_equal(rows(scales, at, page).cpu().numpy(), s, equal_nan=True)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,heads,D,page", [(1, 1, 16, 16), (1, 8, 128, 16), (33, 3, 64, 32), (70, 2, 80, 64),
                                            (100, 5, 128, 16), (257, 1, 256, 128), (40, 2, 208, 1024), (64, 7, 48, 16)])
def test_written_rows_and_no_others(T, heads, D, page, dt, bits):
    pages = (T + page - 1) // page + 3
    cache = new_cache(pages, heads, page, D, bits)
    before = [t.clone() for t in cache]
    k, v = inputs(T, heads, D, dt, T + D)
    g = torch.Generator(device=DEV).manual_seed(D)
    slots = torch.randperm(pages * page, device=DEV, generator=g)[:T]
    if T > 8:
        slots[3] = -1                                        # padding
        slots[7] = pages * page                              # one past the cache
    qa.qa_kv_write(k, v, slots, cache)
    inside = torch.where(slots < pages * page, slots, -1)
    check(cache, k, v, inside, page, bits)
    for t, was in zip(cache, before):
        keep = torch.ones(pages * page, dtype=torch.bool, device=DEV)
        keep[inside[inside >= 0]] = False
        keep = keep.nonzero()[:, 0]
        assert torch.equal(rows(t, keep, page), rows(was, keep, page))
    # and read back, in another order, with places outside the cache
    back = torch.cat([inside.flip(0), torch.tensor([-1, pages * page, -(1 << 40), 1 << 40], device=DEV)])
    for odt in DT.values():
        kr, vr = qa.qa_kv_read(back, cache, out_dtype=odt)
        for got, codes, scales in ((kr, cache[0], cache[1]), (vr, cache[2], cache[3])):
            at = back.clamp(0, pages * page - 1)
            c = rows(codes, at, page)
            c = c.cpu().float() if bits == 8 else torch.from_numpy(unpack(c)).float()
            want = c * rows(scales, at, page).cpu()[..., None]
            want[((back < 0) | (back >= pages * page)).cpu()] = 0.0
            assert torch.equal(got.cpu(), want.to(odt))


@pytest.mark.parametrize("bits", [8, 4])
def test_contiguous_inputs_and_prompts_in_a_row(bits):
    T, heads, D, page = 1000, 4, 128, 64
    cache = new_cache(20, heads, page, D, bits)
    k, v = inputs(T, heads, D, "f16", 5, strided=False)
    slots = torch.arange(T, device=DEV) + 17
    qa.qa_kv_write(k, v, slots, cache)
    check(cache, k, v, slots, page, bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_rows_without_a_finite_scale(dt, bits):
    T, heads, D, page = 9, 2, 64, 16
    cache = new_cache(2, heads, page, D, bits)
    k, v = inputs(T, heads, D, dt, 3)
    k[1, 0, 5] = float("nan")
    k[2, 1, 63] = float("inf")
    v[3, 0, 0] = -float("inf")
    v[4] = 0.0
    if dt != "f16":
        k[5] *= 1e-37                                        # a scale below the normal numbers
        v[5, 1] = torch.finfo(DT[dt]).max
    else:
        k[5] = torch.finfo(torch.float16).smallest_normal / 1024    # the smallest fp16 number
    slots = torch.arange(T, device=DEV)
    qa.qa_kv_write(k, v, slots, cache)
    check(cache, k, v, slots, page, bits)
    assert torch.isnan(cache[1][0, 0, 1]) and torch.isnan(cache[1][0, 1, 2]) and torch.isnan(cache[3][0, 0, 3])
    assert not torch.isnan(cache[1][0, 1, 1]) and (cache[3][0, :, 4] == 1.0).all()
    kr, _ = qa.qa_kv_read(slots, cache, out_dtype=torch.float32)
    assert torch.isnan(kr[1, 0]).all() and torch.isfinite(kr[1, 1]).all()


def test_codes_are_the_row_quantizers():
    """A token's head is a row: the same codes and scales as the library's own row quantizers make."""
    T, heads, D, page = 50, 4, 128, 16
    k, v = inputs(T, heads, D, "f16", 11, strided=False)
    slots = torch.arange(T, device=DEV)
    q, s = qa.qa_quantize_rowwise_int8(k.view(T * heads, D))
    cache = new_cache(4, heads, page, D, 8)
    qa.qa_kv_write(k, v, slots, cache)
    assert torch.equal(rows(cache[0], slots, page), q.view(T, heads, D))
    assert torch.equal(rows(cache[1], slots, page), s.view(T, heads))
    q, s = qa.qa_hadamard_quant_int4(v.reshape(T * heads, D), 1, per_group=False)
    cache = new_cache(4, heads, page, D, 4)
    qa.qa_kv_write(k, v, slots, cache)
    assert torch.equal(rows(cache[2], slots, page), q.view(T, heads, D // 8))
    assert torch.equal(rows(cache[3], slots, page), s.view(T, heads))


def test_one_place_read_many_times():
    cache = new_cache(3, 2, 16, 64, 8)
    slots = torch.full((100,), 20, dtype=torch.int64, device=DEV)
    k, v = qa.qa_kv_read(slots, cache)
    assert (k == k[0]).all() and (v == v[0]).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_scales_of_few_digits(bits):
    """Rows of fp32's smallest numbers: the scale is a few of its last steps, so quotients pass q_max and are clipped."""
    heads, D, page = 2, 64, 16
    top = torch.arange(1, 400, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    k = torch.randint(-10 ** 6, 10 ** 6, (top.numel(), heads, D), device=DEV, generator=g) % (top + 1)[:, None, None]
    k[:, :, 9] = -top[:, None]
    k = k.to(torch.int32)
    k = torch.where(k < 0, -k + torch.iinfo(torch.int32).min, k).view(torch.float32)    # so many steps of 2^-149
    cache = new_cache(25, heads, page, D, bits)
    slots = torch.arange(top.numel(), device=DEV)
    qa.qa_kv_write(k, -k, slots, cache)
    check(cache, k, -k, slots, page, bits)


def test_a_cache_without_pages():
    for bits in (8, 4):
        cache = new_cache(0, 2, 16, 64, bits)
        k, v = inputs(5, 2, 64, "f16", 1)
        slots = torch.arange(5, device=DEV)
        qa.qa_kv_write(k, v, slots, cache)
        kr, vr = qa.qa_kv_read(slots, cache)
        assert (kr == 0).all() and (vr == 0).all()


def test_no_tokens():
    cache = new_cache(2, 2, 16, 64, 8)
    before = [t.clone() for t in cache]
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    e = torch.empty(0, 2, 64, dtype=torch.float16, device=DEV)
    qa.qa_kv_write(e, e, none, cache)
    k, v = qa.qa_kv_read(none, cache)
    assert k.shape == v.shape == (0, 2, 64)
    assert all(torch.equal(a, b) for a, b in zip(before, cache))


def test_refusals():
    T, heads, D, page = 6, 2, 64, 16
    cache = new_cache(2, heads, page, D, 8)
    k, v = inputs(T, heads, D, "f16", 1)
    slots = torch.arange(T, device=DEV)
    with pytest.raises(TypeError):
        qa.qa_kv_write(k.double(), v.double(), slots, cache)
    with pytest.raises(TypeError):
        qa.qa_kv_write(k, v.float(), slots, cache)
    with pytest.raises(TypeError):
        qa.qa_kv_write(k, v, slots.int(), cache)
    with pytest.raises(ValueError):
        qa.qa_kv_write(k, v, slots[:3], cache)
    with pytest.raises(ValueError):
        qa.qa_kv_write(k[:, :1], v[:, :1], slots, cache)
    with pytest.raises(ValueError):
        qa.qa_kv_write(k[:3], v, slots[:3], cache)
    with pytest.raises(ValueError):                          # heads behind each other's values
        qa.qa_kv_write(k.transpose(1, 2).contiguous().transpose(1, 2), v, slots, cache)
    with pytest.raises(TypeError):
        qa.qa_kv_write(k, v, slots, (cache[0].float(),) + cache[1:])
    with pytest.raises(ValueError):
        qa.qa_kv_write(k, v, slots, (cache[0], cache[1][:1], cache[2], cache[3]))
    with pytest.raises(qa.QAError):                          # a token stride of 4-byte steps
        x = torch.zeros(T, heads * D + 2, dtype=torch.float16, device=DEV)[:, :heads * D].view(T, heads, D)
        qa.qa_kv_write(x, v, slots, cache)
    with pytest.raises(qa.QAError):                          # pages of 24 tokens
        qa.qa_kv_read(slots, new_cache(2, heads, 24, D, 8))
    with pytest.raises(TypeError):
        qa.qa_kv_read(slots, cache, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        qa.qa_kv_read(slots.view(2, 3), cache)
