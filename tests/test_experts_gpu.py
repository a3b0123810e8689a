"""qa_experts_int8 against its definition in 64 bits."""
import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def dispatch(ids, E):
    flat = ids.reshape(-1).long().cpu()
    order = torch.cat([torch.nonzero(flat == e)[:, 0] for e in range(E)])
    counts = torch.tensor([int((flat == e).sum()) for e in range(E)])
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    order = torch.cat([order, torch.full((flat.numel() - order.numel(),), -1)])
    return order.to(torch.int32).to(DEV), offsets.to(torch.int32).to(DEV)


def make(T, K, F, E, k, ids=None, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + T * 7 + K + F * 3 + E)
    codes = lambda *s: (torch.randn(*s, device=DEV, generator=g) * 32).round().clamp(-127, 127).to(torch.int8)
    rand = lambda *s: torch.rand(*s, device=DEV, generator=g) + 0.5
    if ids is None:
        ids = torch.rand(T, E, device=DEV, generator=g).topk(k, 1).indices.to(torch.int32)
    order, offsets = dispatch(ids, E)
    c = dict(Xq=codes(T, K), s_x=rand(T) / 32, weights=(rand(T, k) / k).masked_fill(ids < 0, 0.0), order=order,
             offsets=offsets, W13=codes(E, 2 * F, K), s13=rand(E, 2 * F) * (1.5 / 32 / K ** 0.5), W2=codes(E, K, F),
             s2=rand(E, K) * (1.0 / 32 / F ** 0.5))
    return c, ids


def check(c, ids, dt="f16", **kw):
    out = qa.qa_experts_int8(**c, out_dtype=DT[dt], **kw)
    T, K = c["Xq"].shape
    E, F = c["W13"].shape[0], c["W2"].shape[2]
    k = ids.shape[1]
    D = torch.float64
    p = {n: t.cpu().to(D) for n, t in c.items() if n not in ("order", "offsets")}
    ids = ids.cpu()
    want, room = torch.zeros(T, K, dtype=D), torch.zeros(T, K, dtype=D)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        gu = (p["Xq"][t] @ p["W13"][e].T) * p["s_x"][t][:, None] * p["s13"][e]
        gt, up = gu[:, :F], gu[:, F:]
        h = gt * torch.sigmoid(gt) * up
        s = h.abs().amax(1) / 127
        s[s == 0] = 1.0
        v = h / s[:, None]
        w = p["weights"][t, j][:, None]
        y = (v.round() @ p["W2"][e].T) * s[:, None] * p["s2"][e]
        # h in fp32 is off by the scales' products, exp (2 units), a quotient and a product, and by |g| 2^-23 through
        # the exponent; s by that of the largest h: codes that lie so near to a tie may differ by one
        tol = (16 + gt.abs().amax()) * 2.0 ** -23
        near = ((v - v.floor() - 0.5).abs() <= 2 * tol * v.abs() + 1e-12).to(D)
        off = (near @ p["W2"][e].abs().T) * s[:, None] * p["s2"][e] + y.abs() * (tol + 8 * 2.0 ** -24)
        want.index_put_((t,), w * y, accumulate=True)
        room.index_put_((t,), w.abs() * off + (w * y).abs() * (k + 2) * 2.0 ** -24, accumulate=True)
    got = out.cpu().to(D)
    assert got.shape == (T, K) and torch.isfinite(got).all()
    assert ((got - want).abs() <= room + ULP[dt] * (want.abs() + room) + TINY[dt]).all()
    none = (ids < 0).all(1)
    assert (got[none] == 0).all()
    return out


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,K,F,E,k", [
    (1, 16, 16, 1, 1), (1, 64, 32, 4, 2), (3, 80, 48, 3, 3), (8, 256, 112, 16, 4), (17, 272, 144, 8, 2),     # weights streamed
    (40, 512, 80, 5, 2), (64, 128, 128, 2, 1), (100, 208, 96, 4, 2),
    (130, 320, 144, 2, 2), (300, 256, 272, 3, 2), (513, 128, 64, 1, 1), (400, 96, 528, 5, 3)])              # tiles
def test_against_64_bits(dt, T, K, F, E, k):
    check(*make(T, K, F, E, k), dt=dt)


@pytest.mark.parametrize("F", [240, 256, 272, 1024, 1040, 2048, 2064, 4096, 4112, 6160])
@pytest.mark.parametrize("T,k", [(3, 2), (37, 1)])
def test_widths_of_the_hidden_rows(T, k, F):
    check(*make(T, 48, F, 2, k), dt="f32")


@pytest.mark.parametrize("T,K,k", [(1, 16, 7), (5, 1040, 8), (3, 4112, 9), (33, 80, 20), (2, 32, 32)])
def test_many_slots_to_a_token(T, K, k):
    ids = torch.rand(T, 32, device=DEV, generator=torch.Generator(device=DEV).manual_seed(k)).topk(k, 1).indices.to(torch.int32)
    ids[:, ::5] = -1
    check(*make(T, K, 32, 32, k, ids=ids), dt="f32")


@pytest.mark.parametrize("T", [20, 600])
def test_uneven_experts(T):
    """Experts without tokens, one that takes nearly all, tokens without experts and half-filled slots."""
    ids = torch.full((T, 2), 3, dtype=torch.int32, device=DEV)
    ids[:, 1] = 5
    ids[::7, 0] = 0
    ids[::5, 1] = -1
    ids[4] = -1
    ids[T - 1] = -1
    check(*make(T, 144, 80, 9, 2, ids=ids))


def test_no_pair_at_all():
    ids = torch.full((70, 2), -1, dtype=torch.int32, device=DEV)
    for T in (5, 70):
        c, i = make(T, 64, 32, 1, 2, ids=ids[:T])
        assert (check(c, i) == 0).all()


def test_rows_of_zeros():
    c, ids = make(9, 64, 32, 3, 2)
    c["Xq"][4] = 0
    out = check(c, ids)
    assert (out[4] == 0).all()


def test_an_infinite_scale_stays_in_its_row():
    for T in (9, 200):
        c, ids = make(T, 64, 32, 2, 2)
        clean = qa.qa_experts_int8(**c)
        c["s_x"][4] = float("nan")
        out = qa.qa_experts_int8(**c)
        assert torch.isnan(out[4]).all()
        keep = torch.arange(T, device=DEV) != 4
        assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("T", [12, 300])
def test_after_routing(T):
    E, k, K, F = 8, 2, 128, 64
    c, _ = make(T, K, F, E, k)
    logits = torch.randn(T, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T))
    logits[3] = -float("inf")
    ids, w, order, offsets = qa.qa_route_experts(logits, k)
    c.update(weights=w, order=order, offsets=offsets)
    check(c, ids)


def test_workspace_of_any_content():
    c, ids = make(150, 128, 64, 2, 2)
    n = qa.qa_experts_int8_workspace(150, 128, 2, 2, 64)
    a = check(c, ids, workspace=torch.zeros(n, dtype=torch.uint8, device=DEV))
    b = check(c, ids, workspace=torch.full((n,), 255, dtype=torch.uint8, device=DEV))
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,K,F,E,k", [(2000, 272, 1552, 2, 2), (1111, 144, 2064, 4, 3), (4100, 96, 1536, 1, 1)])
def test_largest_tiles(T, K, F, E, k):
    """More than 120 rows for each expert and enough tiles of 128 rows for all of the device."""
    assert T * k // E >= 120 and (T * k // 128) * ((2 * F + 191) // 192) >= 512
    check(*make(T, K, F, E, k))


@pytest.mark.parametrize("first,last", [(0, 3), (2, 5), (4, 9), (8, 9)])
@pytest.mark.parametrize("T", [6, 40, 600])
def test_a_part_of_the_experts(T, first, last):
    """The experts that one of several devices holds: their weights and their part of `offsets`, which then starts past 0
    and ends before the last pair.  The other experts' pairs add nothing, whatever the workspace held."""
    c, ids = make(T, 144, 80, 9, 3)
    part = {**c, "offsets": c["offsets"][first:last + 1]}
    for name in ("W13", "s13", "W2", "s2"):
        part[name] = c[name][first:last]
    mine = torch.where((ids >= first) & (ids < last), ids - first, torch.full_like(ids, -1))
    n = qa.qa_experts_int8_workspace(T, 144, 3, last - first, 80)
    check(part, mine, dt="f32", workspace=torch.full((n,), 255, dtype=torch.uint8, device=DEV))


def test_refusals():
    c, _ = make(4, 64, 32, 2, 2)
    with pytest.raises(qa.QAError):
        qa.qa_experts_int8(**c, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    for name in ("s_x", "order", "offsets", "s13", "s2"):
        with pytest.raises(ValueError):
            qa.qa_experts_int8(**{**c, name: c[name][:-1].contiguous()})
    with pytest.raises(TypeError):
        qa.qa_experts_int8(**{**c, "W13": c["W13"].half()})
    with pytest.raises(ValueError):
        qa.qa_experts_int8(**{**c, "W2": c["W2"].transpose(1, 2)})
    bad, _ = make(4, 64, 32, 2, 2)
    bad["Xq"], bad["W13"], bad["W2"] = bad["Xq"][:, :56].contiguous(), bad["W13"][:, :, :56].contiguous(), bad["W2"][:, :56].contiguous()
    bad["s2"] = bad["s2"][:, :56].contiguous()
    with pytest.raises(qa.QAError):
        qa.qa_experts_int8(**bad)                            # K % 16
