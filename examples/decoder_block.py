"""A decoder block's int8 half on packed requests: norm -> shared projection with each request's adapter -> residual
+ norm -> routing -> experts, as a serving program would call them, for prompts and for single tokens.

    python examples/decoder_block.py            # on a GPU; prints both steps' times and their distance from fp32

The projection stands where attention's input and output projections would; attention itself, on a quantized cache, is
in attention_step.py.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_quantized_linear_int8_amd as qa  # noqa: E402


class DecoderBlock:
    """Weights of one block, quantized once: int8 codes and a scale per output channel."""

    def __init__(self, K=1024, F=512, E=16, k=4, adapters=4, rank=16, device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s, std=1.0: torch.randn(*s, device=device, generator=g) * std   # noqa: E731
        self.K, self.F, self.E, self.k = K, F, E, k
        self.g1, self.g2 = (1.0 + n(K, std=0.1)).half(), (1.0 + n(K, std=0.1)).half()
        self.W = n(K, K, std=K ** -0.5).half()
        self.W13, self.W2 = n(E, 2 * F, K, std=K ** -0.5).half(), n(E, K, F, std=F ** -0.5).half()
        self.router, self.bias = n(E, K, std=K ** -0.5).half(), n(E, std=0.02)
        self.A, self.B = n(adapters, rank, K, std=K ** -0.5).half(), n(adapters, K, rank, std=0.05).half()
        self.alpha = torch.full((adapters,), 2.0, device=device)
        self.Wq, self.s_w = qa.qa_quantize_rowwise_int8(self.W)
        q, s = qa.qa_quantize_rowwise_int8(self.W13.view(E * 2 * F, K))
        self.W13q, self.s13 = q.view(E, 2 * F, K), s.view(E, 2 * F)
        q, s = qa.qa_quantize_rowwise_int8(self.W2.view(E * K, F))
        self.W2q, self.s2 = q.view(E, K, F), s.view(E, K)

    def __call__(self, x, residual, seg, which, stream=None):
        """x, residual fp16 [tokens x K]: the last block's output and the running sum; seg i32 [R + 1] the requests'
        token starts, which i32 [R] their adapters -> (output, running sum, the tokens' experts)."""
        codes, s, total, y = qa.qa_rmsnorm_int8(x, self.g1, residual=residual, want_y=True, stream=stream)
        mixed = qa.qa_qlinear_int8_lora(codes, s, y, self.Wq, self.s_w, self.A, self.B, self.alpha, seg, which,
                                        stream=stream)
        codes, s, total, y = qa.qa_rmsnorm_int8(mixed, self.g2, residual=total, want_y=True, total=total, stream=stream)
        logits = y @ self.router.t()
        ids, w, order, offsets = qa.qa_route_experts(logits, self.k, bias=self.bias, score=qa.QA_SCORE_SIGMOID,
                                                   renorm=True, stream=stream)
        return qa.qa_experts_int8(codes, s, w, order, offsets, self.W13q, self.s13, self.W2q, self.s2,
                                  stream=stream), total, ids

    def plain(self, x, residual, seg, which, ids):
        """The same block in fp32 on the unquantized weights, with the given choice of experts -> (output, running
        sum, its own choice)."""
        f = lambda t: t.float()                                                      # noqa: E731
        norm = lambda h, g: h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * f(g)   # noqa: E731
        total = f(x) + f(residual)
        y = norm(total, self.g1)
        mixed = y @ f(self.W).t()
        cuts = seg.tolist()
        for i, a in enumerate(which.tolist()):
            t = slice(cuts[i], cuts[i + 1])
            if a >= 0:
                mixed[t] += self.alpha[a] * (y[t] @ f(self.A[a]).t()) @ f(self.B[a]).t()
        total = total + mixed
        y = norm(total, self.g2)
        s = torch.sigmoid(y @ f(self.router).t())
        own = (s + self.bias).topk(self.k, 1).indices
        ids = ids.long()
        w = s.gather(1, ids)
        w = w / w.sum(1, keepdim=True)
        out = torch.zeros_like(total)
        for e in range(self.E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            gu = y[t] @ f(self.W13[e]).t()
            h = torch.nn.functional.silu(gu[:, : self.F]) * gu[:, self.F:]
            out.index_add_(0, t, w[t, j][:, None] * (h @ f(self.W2[e]).t()))
        return out, total, own


def requests(lengths, adapters, device="cuda:0"):
    """Token starts and adapters of packed requests (every fourth one without an adapter)."""
    seg = torch.tensor([0] + lengths, device=device).cumsum(0).to(torch.int32)
    which = torch.tensor([-1 if i % 4 == 3 else i % adapters for i in range(len(lengths))], device=device)
    return seg, which.to(torch.int32)


def compare(block, lengths, seed=0):
    """Relative distance of the block's output and running sum from fp32 with the same experts, and the share of the
    (token, expert) choices that fp32 makes as well."""
    T = sum(lengths)
    g = torch.Generator(device="cuda:0").manual_seed(1000 + seed)     # not the weights' seed: their draws would agree
    x = torch.randn(T, block.K, device="cuda:0", generator=g).half()
    r = torch.randn(T, block.K, device="cuda:0", generator=g).half()
    seg, which = requests(lengths, block.A.shape[0])
    out, total, ids = block(x, r, seg, which)
    want, want_total, own = block.plain(x, r, seg, which, ids)
    off = lambda a, b: float((a.float() - b).norm() / b.norm())                      # noqa: E731
    same = (ids.long()[:, :, None] == own[:, None, :]).any(2).float().mean()
    return off(out, want), off(total, want_total), float(same)


def main():
    block = DecoderBlock(K=4096, F=1024, E=64, k=8, adapters=8)
    for name, lengths in (("prompts", [700, 1, 0, 333, 1014]), ("single tokens", [1] * 24)):
        rel, rel_total, share = compare(block, lengths)
        x = torch.randn(sum(lengths), block.K, device="cuda:0").half()
        seg, which = requests(lengths, 8)
        for _ in range(5):
            block(x, x, seg, which)
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            block(x, x, seg, which)
        torch.cuda.synchronize()
        print("%s: %d tokens, %.1f us a block; off fp32 by %.3g (sum %.3g), %.1f%% of the experts as in fp32" %
              (name, sum(lengths), (time.perf_counter() - t) / 20 * 1e6, rel, rel_total, 100 * share))


if __name__ == "__main__":
    main()
