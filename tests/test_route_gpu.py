"""qa_route_experts against the definition in 64 bits: choices, weights and the grouping of the pairs."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SCORE = {"softmax": qa.QA_SCORE_SOFTMAX, "sigmoid": qa.QA_SCORE_SIGMOID}


def reference(x, k, bias, score, groups, top_groups, group_top, renorm, scale):
    """One row at a time, in 64 bits -> ids, weights, and whether the row's choice hangs on less than 4e-6."""
    T, E = x.shape
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    close = np.zeros(T, bool)
    for t in range(T):
        v = x[t].astype(np.float64)
        v = np.where(np.isnan(v), -np.inf, np.minimum(v, np.finfo(np.float32).max))
        live = v > -np.inf
        if not live.any():
            continue
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-v))
            else:
                s = np.exp(v - v.max())
                s = s / s.sum()
        by_logit = score == "softmax" and bias is None and (groups == 1 or group_top == 1)
        c = v.copy() if by_logit else s + (0 if bias is None else bias.astype(np.float64))
        c[~live] = -np.inf

        def near(a, first, last):
            """Whether unequal neighbours, from rank `first` to rank `last` from the top, are as near as that."""
            a = -np.sort(-a[np.isfinite(a)])[first:last + 1]
            d = -np.diff(a)
            return not by_logit and bool(((d > 0) & (d < 4e-6 * np.maximum(np.abs(a[1:]), 1e-2))).any())
        if groups > 1:
            g = c.reshape(groups, -1)
            top = -np.sort(-g, 1)[:, :group_top]
            val = np.where(np.isinf(top[:, 0]), -np.inf, np.where(np.isinf(top), 0, top).sum(1))
            close[t] |= near(val, top_groups - 1, top_groups)
            keep = np.argsort(-val, kind="stable")[:top_groups]
            mask = np.ones(groups, bool)
            mask[keep] = False
            c = np.where(np.repeat(mask, E // groups), -np.inf, c)
        close[t] |= near(c, 0, k)
        o = np.argsort(-c, kind="stable")[:k]
        o = o[c[o] > -np.inf]
        ids[t, :len(o)] = o
        w[t, :len(o)] = s[o]
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale, close


def check(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    ids, w, order, offsets = qa.qa_route_experts(logits, k, bias=bias, score=SCORE[score], groups=groups,
                                                 top_groups=top_groups, group_top=group_top, renorm=renorm, scale=scale)
    T, E = logits.shape
    rid, rw, close = reference(logits.float().cpu().numpy(), k, None if bias is None else bias.cpu().numpy(), score,
                               groups, top_groups, group_top, renorm, scale)
    ids, w, order, offsets = (t.cpu().numpy() for t in (ids, w, order, offsets))
    assert close.mean() < 0.2
    assert np.array_equal(ids[~close], rid[~close])
    # exp within 2 units of fp32, a sum of at most 16 + 6 terms a lane and the quotients; an exponent x - max rounds
    # once, by at most |x - max| 2^-24 relative to the result
    tol = (40 + 2 * np.nan_to_num(np.abs(logits.float().cpu().numpy()), posinf=0, neginf=0).clip(0, 100).max()) * 2.0 ** -24
    assert (np.abs(w[~close] - rw[~close]) <= tol * np.abs(rw[~close]) + 1e-37 * scale).all()
    # the grouping, of the ids that came
    flat = ids.reshape(-1)
    want = np.concatenate([np.nonzero(flat == e)[0] for e in range(E)] + [np.full((flat < 0).sum(), -1)])
    assert np.array_equal(order, want)
    assert np.array_equal(offsets, np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]))


def logits_of(T, E, dt, seed=0, std=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed * 7 + T * 1031 + E)
    return (torch.randn(T, E, device=DEV, generator=g) * std).to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 2, 2), (63, 16, 4), (64, 33, 8), (65, 64, 6), (129, 100, 16),
                                   (70, 128, 32), (200, 256, 8), (66, 257, 5), (33, 512, 17), (65, 1000, 32),
                                   (3, 1024, 8)])
def test_against_64_bits(dt, score, T, E, k):
    check(logits_of(T, E, dt), k, score=score)


@pytest.mark.parametrize("renorm,scale", [(False, 1.0), (True, 2.5), (False, 0.5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(100, 64, 6), (40, 255, 8), (30, 700, 8)])
def test_bias(score, T, E, k, renorm, scale):
    g = torch.Generator(device=DEV).manual_seed(E)
    bias = torch.randn(E, device=DEV, generator=g) * 0.2
    check(logits_of(T, E, "f32"), k, bias=bias, score=score, renorm=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("T,E,k,groups,top_groups", [(70, 256, 8, 8, 4), (65, 64, 4, 4, 1), (33, 96, 6, 32, 7),
                                                     (20, 640, 8, 10, 3), (9, 12, 3, 12, 5), (17, 60, 15, 4, 1),
                                                     (40, 128, 8, 8, 8)])
def test_groups(score, bias, group_top, T, E, k, groups, top_groups):
    g = torch.Generator(device=DEV).manual_seed(E + groups)
    b = torch.randn(E, device=DEV, generator=g) * 0.2 if bias else None
    check(logits_of(T, E, "f32", seed=3), k, bias=b, score=score, groups=groups, top_groups=top_groups,
          group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_ties_go_to_the_lower_index(score, groups):
    x = torch.randint(-2, 3, (130, 64), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).float()
    check(x, 8, score=score, groups=groups, top_groups=max(1, groups // 2))
    check(torch.zeros(65, 40, device=DEV), 8, score=score, groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_masked_and_extreme_logits(dt, score, bias, groups, top_groups, group_top):
    x = logits_of(140, 64, dt, seed=5)
    low = torch.finfo(DT[dt]).min
    x[0] = -math.inf                                          # nothing left
    x[1] = float("nan")
    x[2, 3:] = -math.inf                                      # fewer than k left
    x[3, ::2] = float("nan")
    x[4] = low                                                # the type's lowest value everywhere
    x[5, 10:] = low
    x[6, 20] = math.inf
    x[7, 8:24] = -math.inf                                    # two groups of masked experts
    x[8, 1:] = -math.inf
    x[139] = -math.inf                                        # the last token
    b = torch.linspace(-0.3, 0.3, 64, device=DEV) if bias else None
    check(x, 8, bias=b, score=score, groups=groups, top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("E,k,groups", [(64, 8, 1), (64, 8, 8), (64, 20, 1), (600, 8, 1)])
def test_a_bias_that_is_no_number_masks_its_expert(E, k, groups):
    x = logits_of(130, E, "f32", seed=9)
    bias = torch.linspace(-0.2, 0.2, E, device=DEV)
    kw = dict(score=qa.QA_SCORE_SIGMOID, groups=groups, top_groups=max(1, groups // 2), group_top=2)
    low = bias.clone()
    low[::3] = -math.inf
    bias[::3] = float("nan")
    got, want = qa.qa_route_experts(x, k, bias=bias, **kw), qa.qa_route_experts(x, k, bias=low, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (got[0] % 3 != 0).all() or (got[0] < 0).any()
    none = qa.qa_route_experts(x, k, bias=torch.full((E,), float("nan"), device=DEV), **kw)
    assert (none[0] == -1).all() and (none[1] == 0).all() and (none[3] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top_groups", [(70, 16, 16, 1, 1), (66, 31, 9, 1, 1), (65, 128, 12, 1, 1),
                                                     (40, 256, 16, 1, 1), (33, 256, 16, 16, 1), (33, 96, 14, 4, 2),
                                                     (20, 96, 16, 32, 9), (20, 256, 17, 8, 4)])
def test_more_than_eight(score, T, E, k, groups, top_groups):
    x = logits_of(T, E, "f32", seed=11)
    x[1] = -math.inf
    x[2, 5:] = -math.inf                                      # fewer than k left
    x[3, ::2] = float("nan")
    x[4, :E // 2] = x[4, 0]                                   # equal from the bound's place on
    kw = dict(groups=groups, top_groups=top_groups, group_top=2)
    check(x, k, score=score, **kw)
    check(x, k, score=score, bias=torch.linspace(-0.3, 0.3, E, device=DEV), renorm=False, **kw)
    check(torch.randint(-2, 3, (T, E), device=DEV, generator=torch.Generator(device=DEV).manual_seed(E)).float(), k,
          score=score, **kw)


@pytest.mark.parametrize("same", [15, 16, 17, 31, 32, 33, 40])
@pytest.mark.parametrize("k", [8, 12])
def test_so_many_equal_largest(same, k):
    """16 or 32 values at the bound are taken another way than one more."""
    for E in (64, 200):
        x = logits_of(50, E, "f32", seed=same).clamp(-4, 4)
        at = torch.rand(50, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(k)).topk(same, 1).indices
        check(x.scatter(1, at, 6.0), k)


def test_two_infinite_logits_share_the_weight():
    x = torch.zeros(1, 8, device=DEV)
    x[0, 2] = x[0, 5] = math.inf
    ids, w, _, _ = qa.qa_route_experts(x, 3, renorm=False)
    assert ids[0].tolist() == [2, 5, 0] and w[0].tolist() == [0.5, 0.5, 0.0]


@pytest.mark.parametrize("E,k", [(12, 12), (16, 8), (600, 20)])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_scores_far_below_zero(E, k, renorm):
    """Scores down to fp32's smallest number and to 0, chosen through a bias of zeros."""
    x = torch.full((70, E), -300.0, device=DEV)
    steps = torch.linspace(-104.0, -20.0, 70, device=DEV)
    for j in range(min(k, 8)):
        x[:, (5 * j + 3) % E] = steps - 1.25 * j
    kw = dict(score=qa.QA_SCORE_SIGMOID, renorm=renorm)
    ids, w, _, _ = qa.qa_route_experts(x, k, bias=torch.zeros(E, device=DEV), **kw)
    s = torch.sigmoid(x.double())
    picked = s.gather(1, ids.long())
    # a score rounds to fp32's step below its smallest normal number, 2^-149; otherwise the bounds of check()
    unit, rel = 2.0 ** -149, 240 * 2.0 ** -24
    if renorm:
        total = picked.sum(1, keepdim=True)
        none = (picked < unit / 2).all(1)
        near = (total[:, 0] < k * unit)                      # rounded away or not: nothing to compare
        want = torch.where(total > 0, picked / total, picked)
        room = (picked * rel + unit) / total + want * (rel + k * unit / total)
        assert (w[none] == 0).all()
        assert ((w.double() - want).abs() <= room)[~near].all()
    else:
        assert ((w.double() - picked).abs() <= picked * rel + unit).all()
    # the largest first, as far as fp32 tells them apart
    best = s.topk(k, 1).values
    assert ((picked - best).abs() <= best * 2 * rel + 2 * unit).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k,groups", [(64, 8, 1), (64, 20, 1), (600, 8, 1), (128, 8, 4), (100, 6, 10)])
def test_sigmoid_keeps_the_order_of_saturated_logits(E, k, groups, renorm):
    """Logits past 17, where the score is 1 in fp32, and below -104, where it is 0: the largest are chosen all the same."""
    g = torch.Generator(device=DEV).manual_seed(E + k)
    x = torch.empty(70, E, device=DEV)
    for t in range(70):
        p = torch.randperm(E, device=DEV, generator=g).float()
        x[t] = (18 + p, -89 - p / 64, -200 - p, 40 - 3 * p)[t % 4]
    x[2::4, 7] = -90.0
    ids, w, _, _ = qa.qa_route_experts(x, k, score=qa.QA_SCORE_SIGMOID, groups=groups, top_groups=max(1, groups // 2),
                                       renorm=renorm)
    v = x.view(70, groups, -1)
    if groups > 1:
        kept = torch.zeros(70, groups, dtype=torch.bool, device=DEV)
        v = v.masked_fill(~kept.scatter_(1, v.amax(2).topk(groups // 2, 1).indices, True)[:, :, None], -math.inf)
    want = v.reshape(70, E).topk(k, 1)
    assert torch.equal(ids.long(), want.indices)
    s = torch.sigmoid(want.values.double())
    # fp32's step below its smallest normal number, and the bounds of check()
    unit, rel = 2.0 ** -149, 240 * 2.0 ** -24
    if renorm:
        total = s.sum(1, keepdim=True)
        some = total[:, 0] > 1e3 * unit                      # else the scores are 0 in fp32, or lost nearly all digits
        got, ref = w.double()[some], (s / total)[some]
        assert ((got - ref).abs() <= ref * rel + (1 + k * ref) * unit / total[some]).all() and some.sum() > 40
    else:
        assert ((w.double() - s).abs() <= s * rel + unit).all()


def test_strided_logits():
    x = logits_of(100, 200, "f16")
    check(x[:, 3:67], 4)
    check(x[::2, :128], 4)


@pytest.mark.parametrize("T", [4096, 9000])
def test_many_blocks(T):
    check(logits_of(T, 24, "bf16", std=1.0), 3, renorm=False)


@pytest.mark.parametrize("T,E,k,kw", [
    (16385, 24, 3, dict(renorm=False)), (17000, 250, 8, dict(score="sigmoid")),
    (16449, 128, 8, dict(score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2)),
    (16400, 255, 12, dict(groups=5, top_groups=3, group_top=2))])
def test_blocks_of_many_tokens(T, E, k, kw):
    """More than 16384 tokens: 64 of them to a block, the last one ragged; groups inside the lanes and, at 51 experts a
    group, in LDS."""
    x = logits_of(T, E, "f32", seed=2)
    x[T // 2] = -math.inf
    x[T - 1, 2:] = -math.inf
    bias = torch.linspace(-0.2, 0.2, E, device=DEV) if kw.get("bias") else None
    check(x, k, **{**kw, "bias": bias})


@pytest.mark.parametrize("T", [1, 64])
def test_one_block_with_groups_in_lds(T):
    check(logits_of(T, 255, "f32", seed=4), 9, groups=5, top_groups=2, group_top=2)


def test_one_expert_takes_all():
    x = logits_of(3000, 16, "f32") * 0.1
    x[:, 7] = 50.0
    check(x, 1)


def test_no_tokens():
    ids, w, order, offsets = qa.qa_route_experts(torch.empty(0, 16, device=DEV), 4)
    assert ids.shape == (0, 4) and order.shape == (0,) and (offsets.cpu() == 0).all()


def test_the_same_twice():
    x = logits_of(5000, 128, "f32")
    a, b = qa.qa_route_experts(x, 8), qa.qa_route_experts(x, 8)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals():
    x = torch.zeros(4, 16, device=DEV)
    for kw in (dict(k=0), dict(k=17), dict(k=4, groups=3), dict(k=8, groups=4, top_groups=1), dict(k=4, groups=4, top_groups=5),
               dict(k=4, score=2), dict(k=4, group_top=3), dict(k=4, scale=math.inf)):
        with pytest.raises(qa.QAError):
            qa.qa_route_experts(x, **kw)
    with pytest.raises(TypeError):
        qa.qa_route_experts(x.double(), 2)
    with pytest.raises(ValueError):
        qa.qa_route_experts(x, 2, bias=torch.zeros(15, device=DEV))
    with pytest.raises(ValueError):
        qa.qa_route_experts(x.t(), 2)
    with pytest.raises(qa.QAError):
        qa.qa_route_experts(torch.zeros(2, 1025, device=DEV), 2)
