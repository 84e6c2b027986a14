"""A serving loop of one attention layer and the logits projection: trellis-quantized
projections, an 8-bit paged key/value cache, attention over it, accumulated attention
weight, eviction by that weight, and the adjusted greedy choice.

Every step is the same sequence of library calls, whether it carries a prompt or one
token per user; a step of single tokens is captured once as a CUDA graph and replayed,
the lengths and the last tokens living on the device.

    python examples/serve_step.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import synthetic  # noqa: E402
import trellis_quantized_linear_gb300 as tql  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, BITS = 512, 8, 2, 64, 4
VOCAB, VOCAB_STORED = 1000, 1024  # decodable tokens, stored columns


class Linear:
    """A trellis-quantized projection on the GPU."""

    def __init__(self, K, N, seed, max_rows):
        m = synthetic.make_matrix(K, N, BITS, seed=seed)
        self.K, self.N = K, N
        self.trellis, self.su, self.sv = (torch.from_numpy(np.ascontiguousarray(a.view(np.int16) if a.dtype == np.uint16 else a)).cuda()
                                          for a in (m.trellis, m.su, m.sv))
        self.ws = torch.empty(tql.exl3_linear_workspace_bytes(max_rows, K, N, BITS, 384), dtype=torch.uint8, device="cuda")

    def __call__(self, x, y):
        tql.exl3_linear(x, x.shape[0], self.K, self.trellis, BITS, self.N, self.N, self.su, self.sv, y, tql.EXL3_F16, 384, self.ws)
        return y

    def logits(self, x, logits, argmax):
        tql.exl3_logits_masked(x, x.shape[0], self.K, self.trellis, BITS, self.N, self.N, VOCAB, self.su, self.sv, logits, argmax,
                               384, self.ws)


class Layer:
    """The layer, its cache and the sequences that it serves."""

    def __init__(self, n_seqs, max_tokens, max_rows):
        tql.build()
        tql.exl3_init(torch.cuda.current_device())
        dev = dict(device="cuda")
        self.n_seqs, self.pages = n_seqs, -(-max_tokens // tql.EXL3_KV8_BLOCK)
        self.qkv = Linear(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM, 1, max_rows)
        self.proj = Linear(HEADS * DIM, HIDDEN, 2, max_rows)
        self.head = Linear(HIDDEN, VOCAB_STORED, 3, max_rows)
        self.embed = torch.randn((VOCAB, HIDDEN), generator=torch.Generator(device="cuda").manual_seed(4), **dev).half()
        n_pages = 2 * n_seqs * self.pages  # half of them spare: an evicted sequence moves to new pages
        codes = [torch.zeros((n_pages, KV_HEADS, tql.EXL3_KV8_BLOCK, DIM), dtype=torch.float8_e4m3fn, **dev) for _ in range(2)]
        scales = [torch.ones((n_pages, KV_HEADS), **dev) for _ in range(2)]
        weight = torch.zeros((n_pages, KV_HEADS, tql.EXL3_KV8_BLOCK), **dev)
        self.cache = tql.Exl3Kv8Cache(*codes, *scales, weight)
        self.table = torch.arange(n_seqs * self.pages, dtype=torch.int32, **dev).view(n_seqs, self.pages)
        self.spare = self.table + n_seqs * self.pages
        self.kv_len = torch.zeros(n_seqs, dtype=torch.int32, **dev)
        # what was said so far, for the penalties; a row past its last token holds -1, which is ignored
        self.history = torch.full((n_seqs, max_tokens), -1, dtype=torch.int32, **dev)
        self.history_start = torch.arange(n_seqs + 1, dtype=torch.int32, **dev) * max_tokens
        self.repetition = torch.full((n_seqs,), 1.3, **dev)
        self.presence = torch.full((n_seqs,), 0.1, **dev)
        self.frequency = torch.full((n_seqs,), 0.05, **dev)
        self.allowed = torch.full((n_seqs, -(-VOCAB // 32)), -1, dtype=torch.int32, **dev)
        self.logits = torch.empty((n_seqs, VOCAB_STORED), **dev)
        self.token = torch.zeros(n_seqs, dtype=torch.int32, **dev)

    def batch(self, rows):
        """The sequences with `rows` new tokens each, the new tokens counted in kv_len already."""
        start = torch.arange(self.n_seqs + 1, dtype=torch.int32, device="cuda") * rows
        b = tql.Exl3Kv8Batch(self.table, self.kv_len, start, self.n_seqs * rows, rows)
        n = self.n_seqs * rows
        b.work = dict(
            qkv=torch.empty((n, self.qkv.N), dtype=torch.float16, device="cuda"), mixed=torch.empty((n, HEADS * DIM), dtype=torch.float16, device="cuda"),
            out=torch.empty((n, HIDDEN), dtype=torch.float16, device="cuda"), lse=torch.empty((n, HEADS), device="cuda"),
            ws=torch.empty(tql.exl3_kv8_attention_workspace_bytes(self.cache, b, HEADS), dtype=torch.uint8, device="cuda"))
        return b

    def mix(self, batch, x):
        """x: the rows' hidden states. Appends their keys and values and attends."""
        w = batch.work
        qkv = self.qkv(x, w["qkv"])
        q, k, v = (qkv[:, a * DIM:b * DIM] for a, b in ((0, HEADS), (HEADS, HEADS + KV_HEADS), (HEADS + KV_HEADS, HEADS + 2 * KV_HEADS)))
        tql.exl3_kv8_append(self.cache, batch, k, v)
        tql.exl3_kv8_attention(self.cache, batch, q, HEADS, DIM ** -0.5, w["mixed"], w["ws"], softcap=50.0, lse=w["lse"])
        tql.exl3_kv8_weigh(self.cache, batch, q, HEADS, DIM ** -0.5, w["lse"], softcap=50.0)
        return self.proj(w["mixed"], w["out"])

    def choose(self, hidden):
        """The next token of each sequence from its last row's hidden state."""
        self.head.logits(hidden, self.logits, self.token)
        tql.exl3_logits_adjust(self.logits, VOCAB, self.logits, self.token, history=self.history.view(-1), history_start=self.history_start,
                               repetition=self.repetition, presence=self.presence, frequency=self.frequency, allowed=self.allowed)

    def prompt(self, tokens):
        """tokens: n_seqs x rows. Returns the first choice."""
        rows = tokens.shape[1]
        self.history[:, :rows] = tokens
        self.kv_len += rows
        out = self.mix(self.batch(rows), self.embed[tokens.reshape(-1).long()])
        self.choose(out.view(self.n_seqs, rows, HIDDEN)[:, -1].contiguous())

    def step(self, batch):
        """One token per sequence: the last choice goes in, the next comes out. Nothing here depends on the host."""
        self.history.scatter_(1, self.kv_len.long()[:, None], self.token[:, None])
        self.kv_len += 1
        self.choose(self.mix(batch, self.embed[self.token.long()]))

    def evict(self, budget, recent):
        """Cuts every sequence back to its heaviest and latest tokens, in the spare pages."""
        kept = torch.empty((self.n_seqs, KV_HEADS, budget), dtype=torch.int32, device="cuda")
        new_len = torch.empty_like(self.kv_len)
        pages = -(-budget // tql.EXL3_KV8_BLOCK)
        dst = self.spare[:, :pages].contiguous()
        tql.exl3_kv8_evict(self.cache, tql.Exl3Kv8Batch(self.table, self.kv_len), dst, budget, recent, kept, new_len)
        old = self.table.clone()
        self.table[:, :pages], self.table[:, pages:] = dst, self.spare[:, pages:]
        self.spare = old
        self.kv_len.copy_(new_len)
        return kept


def main(steps=24, budget=150, graph=True):
    torch.cuda.set_device(0)
    layer = Layer(n_seqs=3, max_tokens=320, max_rows=600)
    layer.prompt(torch.randint(0, VOCAB, (3, 190), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda())
    said = [layer.token.tolist()]
    batch = layer.batch(1)
    side = torch.cuda.Stream()
    captured = None
    for i in range(steps):
        if i == steps // 2:
            layer.evict(budget, recent=32)
        if not graph or i == 0:
            layer.step(batch)
        else:
            if captured is None:
                torch.cuda.synchronize()
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured, stream=side):
                    layer.step(batch)
            captured.replay()
        said.append(layer.token.tolist())
    status = tql.exl3_get_device_status()
    return said, layer.kv_len.tolist(), status


if __name__ == "__main__":
    said, lengths, status = main()
    for s, tokens in enumerate(zip(*said)):
        print(f"sequence {s} ({lengths[s]} cached tokens): {' '.join(map(str, tokens))}")
    print("device status:", tql.exl3_status_string(status))
