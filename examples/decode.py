"""A decode loop around the routed-expert block: the library's calls as a serving
program makes them, on a small model with random weights.

    python -m examples.decode [--streams 3] [--steps 16]

Each layer: RMSNorm, a 4-bit projection to queries, keys and values (moe_linear),
rotary embedding, the new keys and values into the 8-bit cache (moe_kv_write),
attention over it (moe_attention; every other layer sees a window, all have sink
logits), the 4-bit output projection, RMSNorm, and the experts with their router
(moe_forward).  Then the 4-bit LM head and moe_sample.  Norms, rotation and the
residual sums are plain torch.  Prompts of different lengths go through the same
calls in one batch, then every step adds one token to each stream.
"""
from __future__ import annotations

import argparse

import torch

import bit_moe_decode_02_gb300 as moe


class Model:
    """Sizes after the gpt-oss family's shape, much smaller: grouped query heads of 64, MXFP4 projections and experts."""

    def __init__(self, layers=2, hidden=256, heads=8, kv_heads=2, head_dim=64, experts=8, top_k=2, vocab=1000, streams=3,
                 max_len=512, block=64, window=32, cache_format=moe.MOE_KV_E4M3, seed=0):
        self.layers, self.hidden, self.heads, self.kv_heads, self.head_dim = layers, hidden, heads, kv_heads, head_dim
        self.top_k, self.vocab, self.window, self.block = top_k, vocab, window, block
        g = torch.Generator(device="cuda").manual_seed(seed)
        dev = "cuda"

        def weights(rows, cols, fmt, group, bias):
            codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g, device=dev)
            if fmt == moe.MOE_FMT_MXFP4:
                scales = torch.randint(120, 123, (rows, cols // 32), dtype=torch.uint8, generator=g, device=dev)
            else:
                scales = (torch.rand(rows, cols // group, generator=g, device=dev) * 0.02).half()
            b = (torch.randn(rows, generator=g, device=dev) * 0.1).bfloat16() if bias else None
            return moe.moe_linear_of(codes, scales, b, fmt, group)

        qkv = (heads + 2 * kv_heads) * head_dim
        f4, i4 = moe.MOE_FMT_MXFP4, moe.MOE_FMT_INT4
        self.qkv = [weights(qkv, hidden, f4, 32, True) for _ in range(layers)]
        self.proj = [weights(hidden, heads * head_dim, f4, 32, True) for _ in range(layers)]
        self.head = weights(vocab, hidden, i4, 64, False)
        self.sinks = [torch.randn(heads, generator=g, device=dev) for _ in range(layers)]
        self.embedding = torch.randn(vocab, hidden, generator=g, device=dev)

        # the experts, resident in their own handle
        self.experts = moe.moe_create(hidden, hidden, experts, layers, 64, top_k, f4, 32, 1)
        r = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, generator=g, device=dev)          # noqa: E731
        e = lambda *s: torch.randint(117, 120, s, dtype=torch.uint8, generator=g, device=dev)        # noqa: E731
        n = lambda *s: (torch.randn(*s, generator=g, device=dev) * 0.1).bfloat16()                   # noqa: E731
        for i in range(layers):
            moe.moe_load_experts(self.experts, i, r(experts, 2 * hidden, hidden // 2), e(experts, 2 * hidden, hidden // 32),
                                 n(experts, 2 * hidden), r(experts, hidden, hidden // 2), e(experts, hidden, hidden // 32),
                                 n(experts, hidden))
            moe.moe_load_router(self.experts, i, n(experts, hidden), n(experts))

        # one cache a layer; the streams' blocks are dealt out in advance
        self.ops = moe.moe_ops_create()
        per = -(-max_len // block)
        self.table = torch.arange(streams * per, dtype=torch.int32, device=dev).reshape(per, streams).t().contiguous()
        self.caches = []
        for _ in range(layers):
            codes = torch.zeros(streams * per, kv_heads, 2, block * head_dim, dtype=torch.uint8, device=dev)
            scales = torch.zeros(streams * per, kv_heads, 2, device=dev)
            self.caches.append(moe.moe_kv_cache_of(codes, scales, block, head_dim, cache_format))
        self.lengths = [0] * streams
        half = head_dim // 2
        self.inv_freq = 10000.0 ** (-torch.arange(half, device=dev) / half)

    def close(self):
        torch.cuda.synchronize()
        moe.moe_ops_destroy(self.ops)
        moe.moe_destroy(self.experts)

    @staticmethod
    def _norm(x):
        return (x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def _rotate(self, x, pos):
        a = pos[:, None].float() * self.inv_freq
        c, s = a.cos()[:, None], a.sin()[:, None]
        u, v = x.float().chunk(2, -1)
        return torch.cat((u * c - v * s, v * c + u * s), -1).bfloat16()

    def _linear(self, w, x, out):
        for m in range(0, x.shape[0], 64):                  # moe_linear takes up to 64 tokens
            moe.moe_linear(self.ops, w, x[m:m + 64], out[m:m + 64])
        return out

    def forward(self, tokens):
        """tokens: for each stream a list of new token ids (possibly none).  Logits fp32 of every new token's successor."""
        new = [len(t) for t in tokens]
        before = list(self.lengths)
        self.lengths = [a + b for a, b in zip(before, new)]
        T, dev = sum(new), "cuda"
        cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=dev)
        batch = moe.moe_kv_batch_of(cu, torch.tensor(self.lengths, dtype=torch.int32, device=dev), self.table, T)
        pos = torch.cat([torch.arange(b, b + n, device=dev) for b, n in zip(before, new)])
        x = self.embedding[torch.tensor([t for s in tokens for t in s], device=dev)]          # the residual, fp32
        H, Hk, D = self.heads, self.kv_heads, self.head_dim
        for i in range(self.layers):
            qkv = self._linear(self.qkv[i], self._norm(x), torch.empty(T, (H + 2 * Hk) * D, dtype=torch.bfloat16, device=dev))
            q, k, v = qkv.split((H * D, Hk * D, Hk * D), 1)
            q = self._rotate(q.reshape(T, H, D), pos)
            k = self._rotate(k.reshape(T, Hk, D), pos)
            moe.moe_kv_write(self.ops, self.caches[i], batch, k, v.unflatten(1, (Hk, D)))     # v in the projection's rows
            a = torch.empty_like(q)
            moe.moe_attention(self.ops, self.caches[i], batch, q, a, sinks=self.sinks[i], window=self.window if i % 2 else 0)
            x = x + self._linear(self.proj[i], a.flatten(1), torch.empty(T, self.hidden, device=dev))
            y = x.bfloat16()                                # moe_forward adds to the residual that it is given
            n = self._norm(x)
            for m in range(0, T, 64):
                moe.moe_forward(self.experts, i, n[m:m + 64], None, min(64, T - m), self.top_k, y[m:m + 64])
            x = y.float()
        return self._linear(self.head, self._norm(x), torch.empty(T, self.vocab, device=dev)), cu

    def generate(self, prompts, steps, temperature=0.8, top_k=40, top_p=0.95, min_p=0.02, seed=1):
        """Prompts (lists of ids), then `steps` sampled tokens for each: a list of lists."""
        B, dev = len(prompts), "cuda"
        g = torch.Generator(device=dev).manual_seed(seed)
        f = lambda v: torch.full((B,), v, device=dev)       # noqa: E731
        k = torch.full((B,), top_k, dtype=torch.int32, device=dev)
        token, logprob = torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, device=dev)
        out, feed = [[] for _ in prompts], [list(p) for p in prompts]
        for _ in range(steps):
            logits, cu = self.forward(feed)
            last = logits[(cu[1:] - 1).long()]              # each stream's newest token
            u = torch.rand(B, generator=g, device=dev)
            moe.moe_sample(self.ops, last, f(temperature), k, f(top_p), f(min_p), u, token, logprob)
            feed = [[t] for t in token.tolist()]
            for o, t in zip(out, feed):
                o += t
        if moe.moe_ops_get_status(self.ops) or moe.moe_get_status(self.experts):
            raise RuntimeError(moe.moe_last_error())
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--streams", type=int, default=3)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    model = Model(streams=a.streams)
    prompts = [[(7 * s + 3 * i) % model.vocab for i in range(5 + 20 * s)] for s in range(a.streams)]
    for s, tokens in enumerate(model.generate(prompts, a.steps)):
        print(f"stream {s}: {len(prompts[s])} prompt tokens ->", *tokens)
    model.close()


if __name__ == "__main__":
    main()
