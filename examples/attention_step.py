"""A decoder block's attention half on a quantized cache: norm -> int8 projection to queries, keys and values (bias) ->
keys and values into a paged int8 or int4 cache -> attention -> int8 output projection onto the residual; in chunks of
prompts (the cache's context read back in 16 bits for torch's products) and in steps of one token per sequence.

    python examples/attention_step.py            # on a GPU; prints both parts' times and their distance from fp32
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_quantized_linear_int8_amd as qa  # noqa: E402


class Cache:
    """A paged cache and the pages of its sequences, handed out as they grow."""

    def __init__(self, sequences, pages, heads, page, D, bits, device="cuda:0"):
        width, codes = (D, torch.int8) if bits == 8 else (D // 8, torch.int32)
        new = lambda *s, dt=torch.float32: torch.zeros(pages, heads, page, *s, dtype=dt, device=device)   # noqa: E731
        self.tensors = (new(width, dt=codes), new(), new(width, dt=codes), new())
        self.page, self.free = page, list(range(pages - 1, -1, -1))
        self.pages = [[] for _ in range(sequences)]
        self.lengths = [0] * sequences
        self.device = device

    def grow(self, b, n):
        """Places of n more tokens of sequence b, i64 [n]."""
        first, self.lengths[b] = self.lengths[b], self.lengths[b] + n
        while len(self.pages[b]) * self.page < self.lengths[b]:
            self.pages[b].append(self.free.pop())
        return self.slots(b, first, self.lengths[b])

    def slots(self, b, first, end):
        t = torch.arange(first, end, device=self.device)
        return torch.tensor(self.pages[b], device=self.device)[t // self.page] * self.page + t % self.page

    def table(self):
        """i32 [sequences x most pages] (-1 behind a sequence's last), i32 [sequences] lengths, and the longest."""
        width = max(len(p) for p in self.pages)
        rows = [p + [-1] * (width - len(p)) for p in self.pages]
        i32 = dict(dtype=torch.int32, device=self.device)
        return torch.tensor(rows, **i32), torch.tensor(self.lengths, **i32), max(self.lengths)


class AttentionHalf:
    """Weights of one block's attention, quantized once: int8 codes and a scale per output channel."""

    def __init__(self, K=1024, H=16, heads=4, D=64, device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s, std=1.0: torch.randn(*s, device=device, generator=g) * std    # noqa: E731
        self.K, self.H, self.heads, self.D = K, H, heads, D
        self.g = (1.0 + n(K, std=0.1)).half()
        self.W, self.b = n((H + 2 * heads) * D, K, std=K ** -0.5).half(), n((H + 2 * heads) * D, std=0.1)
        self.Wo = n(K, H * D, std=(H * D) ** -0.5).half()
        self.Wq, self.s_w = qa.qa_quantize_rowwise_int8(self.W)
        self.Woq, self.s_wo = qa.qa_quantize_rowwise_int8(self.Wo)

    def project(self, x, residual, stream=None):
        """-> queries [T x H x D], keys, values [T x heads x D] (views of the projection), the running sum."""
        codes, s, total, _ = qa.qa_rmsnorm_int8(x, self.g, residual=residual, stream=stream)
        y = qa.qa_qlinear_int8_act(codes, s, self.Wq, self.s_w, bias=self.b, stream=stream)
        at, to = self.H * self.D, (self.H + self.heads) * self.D
        split = lambda t: t.unflatten(1, (-1, self.D))                               # noqa: E731
        return split(y[:, :at]), split(y[:, at:to]), split(y[:, to:]), total

    def end(self, o, total, stream=None):
        """The output projection, added to the running sum."""
        codes, s = qa.qa_quantize_rowwise_int8(o.view(-1, self.H * self.D), stream=stream)
        return qa.qa_qlinear_int8_act(codes, s, self.Woq, self.s_wo, residual=total, stream=stream)

    def prompt(self, x, residual, cache, b):
        """A chunk of sequence b's prompt, fp16 [T x K]: attention over all that the cache holds of it, causal."""
        q, k, v, total = self.project(x, residual)
        new = cache.grow(b, x.shape[0])
        qa.qa_kv_write(k, v, new, cache.tensors)
        n, T, group = cache.lengths[b], x.shape[0], self.H // self.heads
        k, v = qa.qa_kv_read(cache.slots(b, 0, n), cache.tensors, out_dtype=torch.float32)
        k, v = (t.repeat_interleave(group, 1).transpose(0, 1).contiguous() for t in (k, v))      # [H x n x D]
        s = q.float().transpose(0, 1).contiguous() @ k.transpose(1, 2).contiguous() * self.D ** -0.5
        late = torch.arange(n, device=x.device) > torch.arange(n - T, n, device=x.device)[:, None]
        o = torch.softmax(s.masked_fill(late, float("-inf")), 2) @ v
        return self.end(o.transpose(0, 1).reshape(T, -1).half(), total)

    def step(self, x, residual, cache, table, lengths, longest, slots, stream=None):
        """One token of every sequence, fp16 [B x K]; its places, the table and the lengths with it included."""
        q, k, v, total = self.project(x, residual, stream)
        qa.qa_kv_write(k, v, slots, cache.tensors, stream=stream)
        o = qa.qa_attn_decode(q, cache.tensors, table, lengths, max_len=longest, stream=stream)
        return self.end(o, total, stream)

    def plain(self, x, residual):
        """One whole sequence in fp32 on the unquantized weights, causal."""
        T, group = x.shape[0], self.H // self.heads
        total = x.float() + residual.float()
        y = total * torch.rsqrt((total * total).mean(1, keepdim=True) + 1e-6) * self.g.float()
        y = (y @ self.W.float().t() + self.b).unflatten(1, (-1, self.D)).transpose(0, 1)
        q, k, v = (t.contiguous() for t in y.split([self.H, self.heads, self.heads]))
        k, v = k.repeat_interleave(group, 0), v.repeat_interleave(group, 0)
        s = q @ k.transpose(1, 2).contiguous() * self.D ** -0.5
        late = torch.ones(T, T, dtype=torch.bool, device=x.device).triu(1)
        o = torch.softmax(s.masked_fill(late, float("-inf")), 2) @ v
        return total + o.transpose(0, 1).reshape(T, -1) @ self.Wo.float().t()


def run(block, lengths, chunk, steps, bits=8, page=16, seed=0):
    """Prompts of the given lengths in chunks, then steps of one token: every output, and fp32's, per sequence."""
    B = len(lengths)
    g = torch.Generator(device="cuda:0").manual_seed(1000 + seed)     # not the weights' seed: their draws would agree
    x, r = ([torch.randn(n + steps, block.K, device="cuda:0", generator=g).half() for n in lengths] for _ in range(2))
    pages = sum(-(-(n + steps) // page) for n in lengths)
    cache = Cache(B, pages, block.heads, page, block.D, bits)
    got = [[] for _ in range(B)]
    for b, n in enumerate(lengths):
        for t in range(0, n, chunk):
            e = min(n, t + chunk)
            got[b].append(block.prompt(x[b][t:e], r[b][t:e], cache, b))
    for i in range(steps):
        slots = torch.cat([cache.grow(b, 1) for b in range(B)])
        xs, rs = (torch.stack([t[b][lengths[b] + i] for b in range(B)]) for t in (x, r))
        out = block.step(xs, rs, cache, *cache.table(), slots)
        for b in range(B):
            got[b].append(out[b:b + 1])
    return [torch.cat(o) for o in got], [block.plain(x[b], r[b]) for b in range(B)]


def main():
    block = AttentionHalf(K=4096, H=32, heads=8, D=128)
    for bits in (8, 4):
        got, want = run(block, [700, 33, 1014], 256, 4, bits=bits)
        off = max(float((a.float() - b).norm() / b.norm()) for a, b in zip(got, want))
        B, n = 24, 4000
        cache = Cache(B, B * 252, block.heads, 16, block.D, bits)
        x = torch.randn(B, block.K, device="cuda:0").half()
        for b in range(B):
            cache.grow(b, n)
        slots = torch.cat([cache.slots(b, n - 1, n) for b in range(B)])
        table = cache.table()
        for _ in range(5):
            block.step(x, x, cache, *table, slots)
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            block.step(x, x, cache, *table, slots)
        torch.cuda.synchronize()
        print("%d bits: off fp32 by %.3g; a step of %d sequences with %d tokens each: %.1f us" %
              (bits, off, B, n, (time.perf_counter() - t) / 20 * 1e6))


if __name__ == "__main__":
    main()
