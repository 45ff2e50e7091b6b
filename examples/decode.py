"""A decode loop around the routed-expert block: the library's calls as a serving
program makes them, on a small model with random weights.

    python -m examples.decode [--streams 3] [--steps 16] [--cache e4m3|int8|mxfp4] [--adapters 2]

Each step begins with moe_kv_plan, which makes the step's batch on the GPU from the
streams' lengths: blocks for the new tokens, their positions.  Each layer: RMSNorm, a
4-bit projection to queries, keys and values (moe_linear) with low-rank adapters of the
streams beside it (moe_lora), rotary positions in place (moe_rope), the new keys and
values into the 8- or 4-bit cache (moe_kv_write), attention over it (moe_attention; every
other layer sees a window, all have sink logits), the 4-bit output projection, RMSNorm,
and the experts with their router (moe_forward).  Then the 4-bit LM head and moe_sample.
Norms and the residual sums are plain torch.  Prompts of different lengths go through the
same calls in one batch, then every step adds one token to each stream.
"""
from __future__ import annotations

import argparse

import torch

import bit_moe_decode_02_gb300 as moe


class Model:
    """Sizes after the gpt-oss family's shape, much smaller: grouped query heads of 64, MXFP4 projections and experts."""

    def __init__(self, layers=2, hidden=256, heads=8, kv_heads=2, head_dim=64, experts=8, top_k=2, vocab=1000, streams=3,
                 max_len=512, block=64, window=32, cache_format=moe.MOE_KV_E4M3, adapters=0, rank=8, seed=0):
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

        # one cache a layer, and the blocks that the streams take from as they grow
        self.ops = moe.moe_ops_create()
        per = -(-max_len // block)
        blocks = streams * per
        self.caches = []
        for _ in range(layers):
            if cache_format == moe.MOE_KV_MXFP4:
                codes, scales = torch.zeros(blocks, kv_heads, 2, block * head_dim * 17 // 32, dtype=torch.uint8, device=dev), None
            else:
                codes = torch.zeros(blocks, kv_heads, 2, block * head_dim, dtype=torch.uint8, device=dev)
                scales = torch.zeros(blocks, kv_heads, 2, device=dev)
            self.caches.append(moe.moe_kv_cache_of(codes, scales, block, head_dim, cache_format))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)                               # noqa: E731
        self.table = torch.full((streams, per), -1, dtype=torch.int32, device=dev)
        self.pool = moe.moe_kv_pool_of(torch.randperm(blocks, generator=g, device=dev).int(), self.table, block)
        self.kv_len, self.state, self.admitted = i32([0] * streams), i32([0, blocks]), i32([0])
        self.lengths = [0] * streams
        self.rope = moe.moe_rope_of(head_dim, 10000.0)
        # adapters of the streams beside the first projection, in turn; the last stream has none
        self.adapter = i32([s % adapters if adapters and s + 1 < streams else -1 for s in range(streams)])
        self.lora = [moe.moe_lora_of(n(adapters, rank, hidden), n(adapters, qkv, rank)) for _ in range(layers)] if adapters else None

    def close(self):
        torch.cuda.synchronize()
        moe.moe_ops_destroy(self.ops)
        moe.moe_destroy(self.experts)

    @staticmethod
    def _norm(x):
        return (x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def _linear(self, w, x, out):
        for m in range(0, x.shape[0], 64):                  # moe_linear takes up to 64 tokens
            moe.moe_linear(self.ops, w, x[m:m + 64], out[m:m + 64])
        return out

    def forward(self, tokens):
        """tokens: for each stream a list of new token ids (possibly none).  Logits fp32 of every new token's successor."""
        new = [len(t) for t in tokens]
        self.lengths = [a + b for a, b in zip(self.lengths, new)]
        T, dev = sum(new), "cuda"
        e = lambda n: torch.empty(n, dtype=torch.int32, device=dev)                                  # noqa: E731
        cu, seq, pos = e(len(new) + 1), e(T), e(T)
        moe.moe_kv_plan(self.ops, self.pool, torch.tensor(new, dtype=torch.int32, device=dev), self.kv_len, self.state, cu, self.kv_len,
                        self.state, self.admitted, seq, pos)
        batch = moe.moe_kv_batch_of(cu, self.kv_len, self.table, T)
        adapter = self.adapter[seq.long()]
        x = self.embedding[torch.tensor([t for s in tokens for t in s], device=dev)]          # the residual, fp32
        H, Hk, D = self.heads, self.kv_heads, self.head_dim
        for i in range(self.layers):
            n = self._norm(x)
            qkv = self._linear(self.qkv[i], n, torch.empty(T, (H + 2 * Hk) * D, dtype=torch.bfloat16, device=dev))
            for m in range(0, T if self.lora else 0, 64):
                moe.moe_lora(self.ops, self.lora[i], adapter[m:m + 64], n[m:m + 64], qkv[m:m + 64])
            q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split((H * D, Hk * D, Hk * D), 1))        # in the projection's rows
            moe.moe_rope(self.ops, self.rope, pos, q, k)
            moe.moe_kv_write(self.ops, self.caches[i], batch, k, v)
            a = torch.empty(T, H, D, dtype=torch.bfloat16, device=dev)
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
    ap.add_argument("--cache", choices=["e4m3", "int8", "mxfp4"], default="e4m3")
    ap.add_argument("--adapters", type=int, default=0)
    a = ap.parse_args()
    cache = dict(e4m3=moe.MOE_KV_E4M3, int8=moe.MOE_KV_INT8, mxfp4=moe.MOE_KV_MXFP4)[a.cache]
    model = Model(streams=a.streams, cache_format=cache, adapters=a.adapters)
    prompts = [[(7 * s + 3 * i) % model.vocab for i in range(5 + 20 * s)] for s in range(a.streams)]
    for s, tokens in enumerate(model.generate(prompts, a.steps)):
        print(f"stream {s}: {len(prompts[s])} prompt tokens ->", *tokens)
    model.close()


if __name__ == "__main__":
    main()
