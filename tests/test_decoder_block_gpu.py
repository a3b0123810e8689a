"""The example decoder block: norm, adapters, routing and experts together, for prompts and for single tokens."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decoder_block", os.path.join(ROOT, "examples", "decoder_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("lengths", [[1], [1] * 9, [5, 0, 1, 40, 17], [300, 0, 1, 128, 77]])
def test_block_against_fp32(example, lengths):
    """int8 codes with absmax scales of K normal values: a step of about 4 / 127 standard deviations, so an error of
    step / sqrt(12) = 0.9% per operand; two operands a product, two products and the norm's codes in a row stay under
    5% of the output."""
    block = example.DecoderBlock(K=512, F=256, E=8, k=2, adapters=3)
    rel, rel_total, share = example.compare(block, lengths, seed=len(lengths))
    assert rel_total < 0.02 and share > 0.8
    assert rel < 0.05


def test_single_tokens_have_the_prompts_sum_and_experts(example):
    """The running sum does not hang on the choice of experts, and the choice on the sums' order for few tokens alone."""
    block = example.DecoderBlock(K=512, F=256, E=8, k=2, adapters=3, seed=3)
    g = torch.Generator(device="cuda:0").manual_seed(5)
    x, r = (torch.randn(130, 512, device="cuda:0", generator=g).half() for _ in range(2))
    seg, which = example.requests([64, 66], 3)
    out, total, ids = block(x, r, seg, which)
    seg1 = torch.tensor([0, 1], dtype=torch.int32, device="cuda:0")
    same = 0
    for t in (0, 63, 64, 129):
        one, sum1, ids1 = block(x[t:t + 1], r[t:t + 1], seg1, which[t // 64:t // 64 + 1] if t < 128 else which[1:2])
        assert (sum1[0].float() - total[t].float()).abs().max() <= 2.0 ** -9 * total[t].float().abs().max()
        if torch.equal(ids1[0], ids[t]):
            same += 1
            assert float((one[0].float() - out[t].float()).norm() / out[t].float().norm()) < 0.02
    assert same >= 3


def test_single_tokens_agree_with_the_prompt(example):
    """A token's output does not hang on the tokens beside it, up to the order of fp32 sums in the forms for few and
    for many tokens."""
    block = example.DecoderBlock(K=512, F=256, E=8, k=2, adapters=3, seed=3)
    g = torch.Generator(device="cuda:0").manual_seed(5)
    T = 130
    x, r = (torch.randn(T, 512, device="cuda:0", generator=g).half() for _ in range(2))
    seg, which = example.requests([64, 66], 3)
    out, total, ids = block(x, r, seg, which)
    for t in (0, 63, 64, 129):
        seg1 = torch.tensor([0, 1], dtype=torch.int32, device="cuda:0")
        one, sum1, ids1 = block(x[t:t + 1], r[t:t + 1], seg1, which[t // 64:t // 64 + 1] if t < 128 else which[1:2])
        if not torch.equal(ids1[0], ids[t]):                 # a choice that hangs on the sums' order
            continue
        assert (sum1[0].float() - total[t].float()).abs().max() <= 2.0 ** -9 * total[t].float().abs().max()
        assert float((one[0].float() - out[t].float()).norm() / out[t].float().norm()) < 0.02
