"""Continuous batching of requests with a small quantized model: requests join with a prompt,
run token by token beside each other, and end; their cache pages come from one pool and go
back to it. A step is of one kind: the prompts that join, while the running requests wait, or
one token of each running request.

A step's lengths, block tables, positions and row ranges are made on the device by
exl3_kv8_plan from one number a sequence. Both kinds of step are the same calls (norm,
projections, rotation, append, attention, MLP); a step of prompts attends over its own keys
and values (exl3_prompt_attention), a step of single tokens over the 8-bit cache, and is
captured once as a CUDA graph, whichever sequences take part in it.

    python examples/serve_requests.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import trellis_quantized_linear_gb300 as tql  # noqa: E402
from serve_step import Linear  # noqa: E402

LAYERS, HIDDEN, INNER, HEADS, KV_HEADS, DIM = 2, 512, 1024, 8, 2, 64
VOCAB, VOCAB_STORED, LONGEST = 1000, 1024, 512
Q, K, V = HEADS * DIM, (HEADS + KV_HEADS) * DIM, (HEADS + 2 * KV_HEADS) * DIM  # column ends of a fused projection


class Engine:
    """The model, its cache pool and `slots` sequences."""

    def __init__(self, slots, pages, max_rows):
        tql.build()
        tql.exl3_init(torch.cuda.current_device())
        g = torch.Generator(device="cuda").manual_seed(4)
        self.slots, self.n_pages, self.max_rows = slots, pages, max_rows

        def weight(n):
            return (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).half()

        self.embed = torch.randn((VOCAB, HIDDEN), generator=g, device="cuda").half()
        self.layers = []
        for i in range(LAYERS):
            codes = [torch.zeros((pages, KV_HEADS, tql.EXL3_KV8_BLOCK, DIM), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
            scales = [torch.ones((pages, KV_HEADS), device="cuda") for _ in range(2)]
            self.layers.append(dict(
                cache=tql.Exl3Kv8Cache(*codes, *scales), norm=weight(HIDDEN), mlp_norm=weight(HIDDEN), q_norm=weight(DIM), k_norm=weight(DIM),
                qkv=Linear(HIDDEN, V, 10 * i + 1, max_rows), proj=Linear(Q, HIDDEN, 10 * i + 2, max_rows), gate=Linear(HIDDEN, INNER, 10 * i + 3, max_rows),
                up=Linear(HIDDEN, INNER, 10 * i + 4, max_rows), down=Linear(INNER, HIDDEN, 10 * i + 5, max_rows)))
        self.norm, self.head = weight(HIDDEN), Linear(HIDDEN, VOCAB_STORED, 99, max(slots, 16))
        angle = torch.arange(LONGEST, device="cuda").double()[:, None] * 1e4 ** (-torch.arange(0, DIM, 2, device="cuda").double() / DIM)
        self.cos_sin = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()

        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device="cuda")

        # one block table for all layers: a sequence's pages have the same numbers in each layer's cache
        self.table, self.kv_len, self.q_start = ints(slots, LONGEST // tql.EXL3_KV8_BLOCK, fill=-1), ints(slots), ints(slots + 1)
        self.free, self.free_count = torch.arange(pages, dtype=torch.int32, device="cuda"), ints(1, fill=pages)
        self.tokens, self.served, self.last = ints(slots), ints(1), ints(slots)
        self.graph = self.step_work = None

    def work(self, rows, longest):
        """Buffers of a step of up to `rows` rows, `longest` of one sequence."""
        def h(n):
            return torch.zeros((rows, n), dtype=torch.float16, device="cuda")

        def i():
            return torch.zeros(rows, dtype=torch.int32, device="cuda")

        w = dict(batch=tql.Exl3Kv8Batch(self.table, self.kv_len, self.q_start, rows, longest), position=i(), slot=i(), stream=h(HIDDEN), normed=h(HIDDEN),
                 qkv=h(V), mixed=h(Q), out=h(HIDDEN), gate=h(INNER), up=h(INNER), inner=h(INNER), logits=torch.zeros((self.slots, VOCAB_STORED), device="cuda"),
                 argmax=torch.zeros(self.slots, dtype=torch.int32, device="cuda"))
        n = tql.exl3_kv8_attention_workspace_bytes(self.layers[0]["cache"], w["batch"], HEADS)
        w["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        return w

    def plan(self, w):
        tql.exl3_kv8_plan(w["batch"], self.tokens, self.kv_len, self.free, self.free_count, self.free_count, self.n_pages, w["position"], w["slot"],
                          self.served)

    def forward(self, w, ids, prompts):
        """ids: the rows' tokens. Leaves each taking-part sequence's next token in self.last."""
        w["stream"].copy_(self.embed[ids.long()])
        added = None  # what the layer before leaves to be added to the stream
        for layer in self.layers:
            tql.exl3_rms_norm(w["stream"] if added is None else added, w["normed"], weight=layer["norm"],
                              residual=None if added is None else w["stream"], residual_out=None if added is None else w["stream"])
            qkv = layer["qkv"](w["normed"], w["qkv"])
            tql.exl3_qk_rotary(qkv, qkv, HEADS, KV_HEADS, DIM, w["position"], self.cos_sin, q_weight=layer["q_norm"], k_weight=layer["k_norm"])
            q, k, v = qkv[:, :Q], qkv[:, Q:K], qkv[:, K:V]
            tql.exl3_kv8_append(layer["cache"], w["batch"], k, v)
            if prompts:
                tql.exl3_prompt_attention(q, k, v, HEADS, KV_HEADS, DIM, self.q_start, DIM ** -0.5, w["mixed"])
            else:
                tql.exl3_kv8_attention(layer["cache"], w["batch"], q, HEADS, DIM ** -0.5, w["mixed"], w["ws"])
            out = layer["proj"](w["mixed"], w["out"])
            tql.exl3_rms_norm(out, w["normed"], weight=layer["mlp_norm"], residual=w["stream"], residual_out=w["stream"])
            tql.exl3_silu_mul(layer["gate"](w["normed"], w["gate"]), layer["up"](w["normed"], w["up"]), w["inner"])
            added = layer["down"](w["inner"], w["out"])
        tql.exl3_rms_norm(added, w["normed"], weight=self.norm, residual=w["stream"], residual_out=w["stream"])
        here = self.q_start[1:] > self.q_start[:-1]
        rows = (self.q_start[1:].long() - 1).clamp(min=0)
        self.head.logits(w["normed"][rows], w["logits"], w["argmax"])
        self.last.copy_(torch.where(here, w["argmax"], self.last))

    def prompts(self, joining):
        """joining: {slot: prompt tokens}. One step of their prompts; the others wait."""
        self.tokens.zero_()
        for slot, ids in joining.items():
            self.tokens[slot] = len(ids)
        ids = torch.tensor([t for slot in sorted(joining) for t in joining[slot]], device="cuda")
        w = self.work(len(ids), max(len(p) for p in joining.values()))
        self.plan(w)
        self.forward(w, ids, True)
        return w

    def ended(self, slots):
        """Gives the pages of these slots back."""
        self.tokens.zero_()
        self.tokens[list(slots)] = -1
        self.plan(self.work(0, 0))

    def _single(self):
        w = self.step_work
        self.plan(w)
        # a row's sequence: the first that ends after it (rows of none take the last one's token and are not used)
        row = torch.arange(self.slots, dtype=torch.int32, device="cuda")
        seq = torch.searchsorted(self.q_start[1:], row, right=True).clamp(max=self.slots - 1)
        self.forward(w, self.last[seq], False)

    def step(self, running, graph=True):
        """The next token of each of the running slots."""
        self.tokens.zero_()
        self.tokens[list(running)] = 1
        if self.step_work is None:
            self.step_work = self.work(self.slots, 1)
        if not graph:
            return self._single()
        if self.graph is None:
            keep = [t.clone() for t in self._state()]
            self._single()  # outside a capture first: what the libraries set up at their first call
            for t, k in zip(self._state(), keep):
                t.copy_(k)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._single()
        self.graph.replay()

    def _state(self):
        return [self.table, self.kv_len, self.q_start, self.free, self.free_count, self.last] + [t for layer in self.layers for t in layer["cache"]._keep if t is not None]


def main(graph=True, slots=4, pages=24, requests=7):
    """Serves requests of different lengths; returns their tokens, the free pages at the end and the device status."""
    torch.cuda.set_device(0)
    e = Engine(slots, pages, 512)
    g = torch.Generator().manual_seed(1)
    waiting = [(torch.randint(0, VOCAB, (20 + 37 * i % 190,), generator=g).tolist(), 5 + 11 * i % 17) for i in range(requests)]
    said, owner, todo = [[] for _ in waiting], {}, {}
    at = 0
    while at < len(waiting) or owner:
        joining = {}
        for slot in range(slots):
            if slot not in owner and at < len(waiting):
                joining[slot], todo[slot], owner[slot] = waiting[at][0], waiting[at][1], at
                at += 1
        if joining:
            e.prompts(joining)
        else:
            e.step(owner, graph)
        if e.served.item() != slots:
            raise RuntimeError("the pool is too small for the requests")
        took_part = joining or owner
        last = e.last.tolist()
        for slot in list(took_part):
            said[owner[slot]].append(last[slot])
            todo[slot] -= 1
        done = [slot for slot in owner if todo[slot] == 0]
        if done:
            e.ended(done)
            for slot in done:
                del owner[slot]
    return said, e.free_count.item(), tql.exl3_get_device_status()


if __name__ == "__main__":
    said, free, status = main()
    for i, tokens in enumerate(said):
        print(f"request {i}: {' '.join(map(str, tokens))}")
    print(f"free pages: {free}; device status: {tql.exl3_status_string(status)}")
