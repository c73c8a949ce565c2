"""A hybrid decoder on the library's operators: a linear-attention layer and a paged-attention layer, each
followed by grouped INT4 experts, over requests of their own lengths.

    python examples/hybrid_decode.py [--requests 4] [--new 8]

Prompts and single tokens go through the same `forward`: page tables and slots for the new tokens
(`page_tables`), keys and values into the cache (`paged_kv_write`), attention over it (`paged_attention`, a
row for every new token with the length that it sees), linear attention (`linear_attention` for prompts,
`linear_attention_step` for single tokens), and INT4 products for the projections, the experts and the
head. Weights are random; there are no position codes, as positions enter through the decays and the mask.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_int4_w4a16_amd as w  # noqa: E402


class HybridDecoder:
    def __init__(self, hidden=512, heads=8, kv_heads=2, dim=64, experts=8, inner=256, topk=2, vocab=1000,
                 pages=256, page_size=16, requests=4, longest=512, seed=0, cache_type=torch.bfloat16):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.topk, self.page_size = heads, kv_heads, dim, topk, page_size
        self.embed = torch.randn(vocab, hidden, device="cuda", generator=self.gen).to(torch.bfloat16)
        self.linear_in = self.int4(3 * heads * dim, hidden)                   # q, k, v
        self.gate = torch.randn(hidden, heads, device="cuda", generator=self.gen) * hidden ** -0.5
        self.linear_out = self.int4(hidden, heads * dim)
        self.attend_in = self.int4((heads + 2 * kv_heads) * dim, hidden)      # q, k, v
        self.attend_out = self.int4(hidden, heads * dim)
        self.router = [torch.randn(hidden, experts, device="cuda", generator=self.gen) for _ in range(2)]
        self.gate_up = [self.int4(2 * inner, hidden, experts) for _ in range(2)]
        self.down = [self.int4(hidden, inner, experts) for _ in range(2)]
        self.head = self.int4(vocab, hidden)
        shape = (pages, kv_heads, page_size, dim)
        self.k_cache, self.v_cache = (torch.zeros(shape, device="cuda").to(cache_type).permute(0, 2, 1, 3)
                                      for _ in range(2))
        self.scales = {}
        if cache_type == torch.float8_e4m3fn:
            self.scales = dict(k_scale=torch.full((kv_heads,), 0.02, device="cuda"),
                               v_scale=torch.full((kv_heads,), 0.02, device="cuda"))
        self.table = torch.full((requests, -(-longest // page_size)), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, device="cuda", generator=self.gen).to(torch.int32)
        self.rank = torch.arange(pages, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.state = torch.zeros(requests, heads, dim, dim, device="cuda")

    def int4(self, rows, cols, experts=None):
        """A random matrix (or one for each expert) in the packed INT4 format."""
        x = torch.randn((experts or 1) * rows, cols, device="cuda", generator=self.gen) * cols ** -0.5
        q, s = w.quantize_pack(x.to(torch.bfloat16))
        return (q, s) if experts is None else (q.view(experts, rows, -1), s.view(experts, rows, -1))

    @staticmethod
    def product(weight, x):
        """x W^T for any number of tokens, 16 at a time; bfloat16."""
        return torch.cat([w.gemv_batched(*weight, x[i:i + 16].contiguous()) for i in range(0, x.shape[0], 16)]
                         ).to(torch.bfloat16)

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def experts(self, layer, x):
        weights, ids = torch.topk(torch.softmax(x.float() @ self.router[layer], -1), self.topk)
        ids = ids.to(torch.int32)
        rows = []
        for t in range(x.shape[0]):
            h = w.moe_gemv_swiglu(*self.gate_up[layer], ids[t], x[t])
            rows.append(w.moe_down_combine(*self.down[layer], ids[t], weights[t], h))
        return torch.stack(rows).to(torch.bfloat16)

    def place(self, new, max_tokens):
        """Pages and slots of a step's new tokens; lengths and the free list move on, all on the device."""
        step = w.page_tables(self.lens, new, self.table, self.free, self.page_size, max_tokens=max_tokens)
        self.lens.copy_(step.seq_lens)
        at = self.rank + step.counts[1]   # what is left, -1 (no page) behind it
        self.free.copy_(torch.where(at < self.free.numel(), self.free[at.clamp(max=self.free.numel() - 1)], -1))
        return step

    def forward(self, tokens, new_lens):
        """Logits of every new token: `tokens` holds new_lens[b] of request b, one after the other."""
        T, heads, kv, dim = tokens.shape[0], self.heads, self.kv_heads, self.dim
        new = torch.tensor(new_lens, dtype=torch.int32, device="cuda")
        step = self.place(new, T)
        row = torch.repeat_interleave(torch.arange(len(new_lens), device="cuda"), new.long())
        x = self.embed[tokens]

        y = self.norm(x)
        q, k, v = self.product(self.linear_in, y).view(T, 3 * heads, dim).split(heads, 1)
        q, k = (torch.nn.functional.normalize(z.float(), dim=-1).to(torch.bfloat16) for z in (q, k))
        decay = torch.nn.functional.logsigmoid(y.float() @ self.gate + 3.0)
        if max(new_lens) == 1 and min(new_lens) == 1:
            o = w.linear_attention_step(q, k, v, decay, self.state)
        else:
            o, _ = w.linear_attention(q, k, v, decay, cu_seqlens=step.cu_new, state=self.state,
                                      state_out=self.state)
        x = x + self.product(self.linear_out, o.reshape(T, -1))
        x = x + self.experts(0, self.norm(x))

        y = self.product(self.attend_in, self.norm(x)).view(T, heads + 2 * kv, dim)
        w.paged_kv_write(y[:, heads:heads + kv], y[:, heads + kv:], self.k_cache, self.v_cache, step.slot_map,
                         **self.scales)
        o = w.paged_attention(y[:, :heads], self.k_cache, self.v_cache, self.table[row], step.positions + 1,
                              **self.scales)
        x = x + self.product(self.attend_out, o.reshape(T, -1))
        x = x + self.experts(1, self.norm(x))
        return self.product(self.head, self.norm(x))

    def generate(self, prompts, count):
        """Greedy continuation of every prompt by `count` tokens; returns the tokens [requests, count]."""
        lens = [len(p) for p in prompts]
        logits = self.forward(torch.cat(prompts), lens)
        last = torch.cumsum(torch.tensor(lens, device="cuda"), 0) - 1
        out = [logits[last].argmax(-1)]
        for _ in range(count - 1):
            out.append(self.forward(out[-1], [1] * len(prompts)).argmax(-1))
        return torch.stack(out, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--new", type=int, default=8)
    ap.add_argument("--e4m3", action="store_true", help="keep keys and values in 8 bits")
    a = ap.parse_args()
    model = HybridDecoder(requests=a.requests, cache_type=torch.float8_e4m3fn if a.e4m3 else torch.bfloat16)
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1000, (5 + 37 * i % 60,), generator=gen).cuda() for i in range(a.requests)]
    for p, t in zip(prompts, model.generate(prompts, a.new).tolist()):
        print(f"prompt of {len(p)} tokens -> {t}")


if __name__ == "__main__":
    main()
