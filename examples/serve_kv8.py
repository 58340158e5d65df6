"""Serving a small decoder on the 8-bit paged KV cache, from prompt to compaction.

A decoder of random weights (hidden 2048, 8 query heads of 256 on one KV head,
feed-forward 8192: the shapes of the package's decoder layer) serves a few
chats through the library's calls:

  1. prompts of different lengths, packed: norm + int8 codes, the fused q/k/v
     linear, prompt_attention, kv8_append into pages;
  2. decode steps for all chats at once: decode_attention_kv8 on the pages;
  3. a chat forked: two answers that share the pages of its past;
  4. a chat that goes on with several new tokens: its past is read back with
     kv8_read and prompt_attention sees past and new tokens;
  5. a chat ended, the cache compacted, and the others carried on.

Every layer has its own cache, all with the same page table.  Run it on a GPU:

  python examples/serve_kv8.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int4_weight_quantized_gb300 as w4
from int4_weight_quantized_gb300 import workloads as wl


class Decoder:
    """Decoder layers of random int4 weights; the embedding is its own output head."""

    def __init__(self, layers=2, hidden=2048, heads=8, kv_heads=1, dim=256, ffn=8192, vocab=4096, seed=0):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim

        def linear(n, k, i):
            # scales that keep a unit-variance input at unit variance
            s = 1.0 / (4.6 * k ** 0.5)
            codes, scales = wl.make_weights_on("cuda", n, k, seed * 1000 + i, 0.7 * s, 1.3 * s)
            return w4.pack(codes), scales
        self.layers = []
        for i in range(layers):
            self.layers.append(dict(qkv=linear((heads + 2 * kv_heads) * dim, hidden, 10 * i),
                                    o=linear(hidden, heads * dim, 10 * i + 1), gate_up=linear(2 * ffn, hidden, 10 * i + 2),
                                    down=linear(hidden, ffn, 10 * i + 3)))
        self.gamma = torch.ones(hidden, dtype=torch.float16, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embedding = torch.randn((vocab, hidden), generator=g, device="cuda", dtype=torch.float16)

    def step(self, tokens, attend):
        """Logits of `tokens` [n]; attend(layer, q, k, v) -> attention output [n][heads][dim]."""
        n, D = tokens.shape[0], self.dim
        x, delta = self.embedding[tokens], None
        for i, w in enumerate(self.layers):
            r = torch.empty_like(x)
            codes, sx = w4.rmsnorm_quant(x, self.gamma, residual=delta, residual_out=r)
            qkv = w4.linear_q8(codes, sx, *w["qkv"]).view(n, self.heads + 2 * self.kv_heads, D)
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)       # parts of one tensor
            a = w4.linear(attend(i, q, k, v).view(n, self.heads * D), *w["o"])
            x, y = torch.empty_like(r), torch.empty_like(r)
            w4.rmsnorm_quant(r, self.gamma, residual=a, residual_out=x, y_out=y)
            delta = w4.linear(w4.linear_gated(y, *w["gate_up"], act=w4.ACT_GELU_TANH), *w["down"])
        return (x + delta).float() @ self.embedding.float().T


class Server:
    """Chats in rows of one page table; a cache for each layer."""

    def __init__(self, model, rows=8, pages=64, page_tokens=64, max_pages=16):
        self.model, self.T = model, page_tokens
        self.caches = [w4.kv8_cache(pages, model.kv_heads, page_tokens, model.dim) for _ in model.layers]
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")

    def _reserve(self, row, tokens):
        """Free pages for `tokens` more tokens of a row (the host knows the lengths here)."""
        have, want = -(-int(self.lens[row]) // self.T), -(-(int(self.lens[row]) + tokens) // self.T)
        if want > have:
            free, count = w4.kv8_free_pages(self.caches[0], self.table, self.lens)
            assert int(count) >= want - have, "the cache is full"
            self.table[row, have:want] = free[:want - have]
            self.lens[row] = min(want * self.T, int(self.lens[row]) + tokens)        # so that they count as held

    def prompt(self, rows, prompts):
        """New tokens (lists) for some rows, behind whatever they hold: logits behind each row's last."""
        start = self.lens[rows].clone()
        for row, p in zip(rows, prompts):
            self._reserve(row, len(p))
        n = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        cu = torch.nn.functional.pad(n.cumsum(0), (1, 0)).int()
        cu_all = torch.nn.functional.pad((start + n).cumsum(0), (1, 0)).int()
        table, total = self.table[rows].contiguous(), int(cu_all[-1])
        fresh = int(start.sum()) == 0

        def attend(i, q, k, v):
            w4.kv8_append(self.caches[i], k, v, table, start, cu)
            if fresh:
                return w4.prompt_attention(q, k, v, cu)
            past = w4.kv8_read(self.caches[i], table, cu_all, total)                 # and the new tokens, as stored
            return w4.prompt_attention(q, *past, cu, cu_all)
        logits = self.model.step(torch.tensor(sum(prompts, []), device="cuda"), attend)
        self.lens[rows] = start + n
        return logits[cu[1:].long() - 1]

    def decode(self, rows, tokens):
        """One token for each of some rows: logits [rows][vocab]."""
        start = self.lens[rows].clone()
        for row in rows:
            self._reserve(row, 1)
        table, lens = self.table[rows].contiguous(), start + 1
        cu = torch.arange(len(rows) + 1, dtype=torch.int32, device="cuda")

        def attend(i, q, k, v):
            w4.kv8_append(self.caches[i], k, v, table, start, cu)
            return w4.decode_attention_kv8(q.contiguous(), self.caches[i], table, lens)
        logits = self.model.step(torch.as_tensor(tokens, device="cuda"), attend)
        self.lens[rows] = lens
        return logits

    def fork(self, src, dst):
        free, _ = w4.kv8_free_pages(self.caches[0], self.table, self.lens)
        s, d = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (src, dst))
        for cache in self.caches:
            w4.kv8_fork(cache, self.table, self.lens, s, d, free[:1])

    def end(self, row):
        self.lens[row] = 0

    def compact(self):
        """The held pages to the front; returns their number."""
        for cache in self.caches:
            table, held = w4.kv8_compact(cache, self.table, self.lens)
        self.table = table
        return int(held)


def main(layers=2, steps=8, say=print):
    model = Decoder(layers)
    server = Server(model)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 4096, (n,), generator=g).tolist() for n in (150, 7, 90)]
    rows = [0, 1, 2]
    logits = server.prompt(rows, prompts)
    said = [list(p) for p in prompts]
    for _ in range(steps):
        tokens = logits.argmax(1)
        for s, t in zip(said, tokens.tolist()):
            s.append(t)
        logits = server.decode(rows, tokens)
    say(f"decoded {steps} tokens behind prompts of {[len(p) for p in prompts]}")

    # the same tokens as one prompt: the cache only rounds keys and values to 8 bits
    check = Server(model)
    whole = check.prompt(rows, said)
    near = torch.nn.functional.cosine_similarity(whole, logits, dim=1)
    say("cosine of the logits with those of the whole sequence as one prompt: " + ", ".join(f"{x:.4f}" for x in near.tolist()))

    server.fork(0, 3)
    one = server.decode([0, 3], [5, 5])
    two = server.decode([0, 3], [17, 18])
    say(f"forked: the same token gives the same logits ({bool(torch.equal(one[0], one[1]))}), "
        f"another token others ({not bool(torch.equal(two[0], two[1]))})")

    more = server.prompt([1], [[9, 8, 7, 6, 5]])
    say(f"a chat went on with 5 tokens behind {int(server.lens[1]) - 5}; its next token is {int(more.argmax())}")

    server.end(2)
    before = server.decode([0, 1, 3], [3, 3, 3])
    held = server.compact()
    same = Server(model)
    same.caches, same.table, same.lens = server.caches, server.table, server.lens - torch.tensor(
        [1, 1, 0, 1, 0, 0, 0, 0], dtype=torch.int32, device="cuda")
    after = same.decode([0, 1, 3], [3, 3, 3])       # the last step again, on the moved pages
    say(f"compacted to {held} pages; the last step again gives the same logits ({bool(torch.equal(before, after))})")
    return dict(near=near, forked_equal=torch.equal(one[0], one[1]), forked_other=not torch.equal(two[0], two[1]), held=held,
                compacted_equal=torch.equal(before, after), status=w4.get_device_status(),
                front=int(server.table.max()) == held - 1)


if __name__ == "__main__":
    main()
