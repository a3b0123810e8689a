"""The operators of a layer's attention half together, as the example uses them: projection, cache, attention, output
projection; prompts in chunks and single tokens, on streams, in replayed graphs and in two calls at once."""
import importlib.util
import os

import pytest
import torch

import bit_quantized_linear_int8_amd as qa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_step", os.path.join(ROOT, "examples", "attention_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits,limit", [(8, 0.02), (4, 0.12)])
@pytest.mark.parametrize("lengths,chunk", [([1], 16), ([5, 64, 33], 16), ([130, 1, 300], 100)])
def test_against_fp32(example, lengths, chunk, bits, limit):
    """A code's step is the row's largest over 127 or 7: of about 3 standard deviations of 64 values, so its error is
    step / sqrt(12) = 0.7% or 12% of a value.  int8: codes of the norm, two weights, keys, values and of the attention's
    output, each under 1%, sums to under 2% of the attention's part, which is smaller than the sum that it is added to.
    int4: 12% of the values, and of the keys in the scores' differences, half of it left where softmax averages
    over tokens; the attention's part is at most about the size of the sum's."""
    block = example.AttentionHalf(K=512, H=8, heads=2, D=64, seed=1)
    got, want = example.run(block, lengths, chunk, 3, bits=bits)
    for a, b in zip(got, want):
        assert a.shape == b.shape
        assert float((a.float() - b).norm() / b.norm()) < limit


def test_single_tokens_agree_with_the_prompt(example):
    """The same tokens in one chunk and one at a time: the cache holds the same codes where the projections agree, and
    the outputs differ by the order of sums and fp16's roundings (2^-11 each of the parts' size)."""
    block = example.AttentionHalf(K=512, H=8, heads=2, D=64, seed=2)
    g = torch.Generator(device=DEV).manual_seed(3)
    x, r = (torch.randn(40, 512, device=DEV, generator=g).half() for _ in range(2))
    one, two = (example.Cache(1, 4, 2, 16, 64, 8) for _ in range(2))
    want = block.prompt(x, r, one, 0)
    for t in range(40):
        slots = two.grow(0, 1)
        got = block.step(x[t:t + 1], r[t:t + 1], two, *two.table(), slots)
        assert float((got[0].float() - want[t].float()).norm() / want[t].float().norm()) < 0.01


def layer(example, B, n, bits, seed=4, **kw):
    """A block, a filled cache and one step's operands, with everything made up front."""
    block = example.AttentionHalf(seed=seed, **kw)
    cache = example.Cache(B, B * (-(-(n + 8) // 16)), block.heads, 16, block.D, bits)
    g = torch.Generator(device=DEV).manual_seed(seed)
    for b in range(B):
        m = max(0, n - 7 * b)
        if m:
            k, v = (torch.randn(m, block.heads, block.D, device=DEV, generator=g).half() for _ in range(2))
            qa.qa_kv_write(k, v, cache.grow(b, m), cache.tensors)
    slots = torch.cat([cache.grow(b, 1) for b in range(B)])
    x, r = (torch.randn(B, block.K, device=DEV, generator=g).half() for _ in range(2))
    return block, cache, x, r, cache.table(), slots


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("B,n", [(1, 3000), (5, 500), (20, 90)])
def test_streams_and_graph_replays(example, B, n, bits):
    block, cache, x, r, table, slots = layer(example, B, n, bits)
    step = lambda stream=None: block.step(x, r, cache, *table, slots, stream=stream)     # noqa: E731
    want = step().clone()
    held = [t.clone() for t in cache.tensors]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(step(), want), i                  # eager work between the replays
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, cache.tensors))


def test_a_graph_of_a_step_goes_on_with_the_sequences(example):
    """One captured step, replayed for the next tokens: lengths, places, tables and inputs change in their buffers."""
    B, n = 4, 100
    block, cache, x, r, table, slots = layer(example, B, n, 8)
    tab = torch.full((B, 16), -1, dtype=torch.int32, device=DEV)
    tab[:, :table[0].shape[1]] = table[0]
    lengths = table[1].clone()
    graph = torch.cuda.CUDAGraph()
    block.step(x, r, cache, tab, lengths, 256, slots)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = block.step(x, r, cache, tab, lengths, 256, slots)
    other = example.Cache(B, len(cache.tensors[0]), block.heads, 16, block.D, 8)
    other.tensors = tuple(t.clone() for t in cache.tensors)
    g = torch.Generator(device=DEV).manual_seed(9)
    for i in range(5):
        new = torch.cat([cache.grow(b, 1) for b in range(B)])
        t, l, most = cache.table()
        x.copy_(torch.randn(B, block.K, device=DEV, generator=g))
        tab[:, :t.shape[1]] = t
        lengths.copy_(l)
        slots.copy_(new)
        graph.replay()
        want = block.step(x, r, other, tab, l, 256, new)     # the same split of the work: the same bits
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
    assert all(torch.equal(a, b) for a, b in zip(other.tensors, cache.tensors))


def test_two_calls_at_once(example):
    """Two streams, two caches, workspaces of their own: each gives what it gives alone."""
    calls, want = [], []
    for i in range(2):
        block, cache, x, r, table, slots = layer(example, 3, 2000 + 500 * i, 8 - 4 * i, seed=10 + i)
        q = torch.randn(3, block.H, block.D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(i))
        calls.append((q, cache.tensors) + table[:2])
        want.append(qa.qa_attn_decode(*calls[i], max_len=table[2]))
        calls[i] = calls[i], table[2]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(qa.qa_attn_decode(*calls[i][0], max_len=calls[i][1], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_graphs_that_share_a_workspace(example):
    """Two captured graphs on one workspace, replayed one after the other: nothing in it has to last from call to call."""
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    made = []
    for i in range(2):
        block, cache, x, r, table, slots = layer(example, 2 + 3 * i, 1500, 8, seed=20 + i)
        q = torch.randn(2 + 3 * i, block.H, block.D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(i)).half()
        f = lambda q=q, c=cache.tensors, t=table: qa.qa_attn_decode(q, c, t[0], t[1], max_len=t[2], workspace=ws)   # noqa: E731
        want = f().clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f()
        made.append((graph, out, want))
    for i in range(6):
        graph, out, want = made[i % 2]
        out.fill_(0)
        ws.fill_(255)                                        # what an earlier call left: NaNs
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_linear_on_streams_and_in_graphs():
    g = torch.Generator(device=DEV).manual_seed(30)
    codes = lambda *s: torch.randint(-127, 128, s, device=DEV, generator=g).to(torch.int8)   # noqa: E731
    for M, K, N in [(4, 512, 640), (12, 4608, 5000), (300, 512, 640)]:      # the three forms
        Xq, Wq, s_x, s_w = codes(M, K), codes(N, K), torch.rand(M, device=DEV), torch.rand(N, device=DEV) / 1000
        b, res = torch.randn(N, device=DEV), torch.randn(M, N, device=DEV).bfloat16()
        f = lambda stream=None: qa.qa_qlinear_int8_act(Xq, s_x, Wq, s_w, bias=b, act=qa.QA_ACT_GELU, residual=res,   # noqa: E731
                                                       stream=stream)
        want = f().clone()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = f(side)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f()
        for i in range(3):
            out.fill_(0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(f(), want)
