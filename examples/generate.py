"""Several continuations of each prompt, end to end through this library: the
prompt's pages are shared, the pages that a continuation writes into are copied
first, ended sequences give theirs back, and the pool is compacted.

    python examples/generate.py [--prompts 4] [--ways 4] [--prompt 500] [--steps 64] [--layers 4] [--vocab 32000]

Random weights: decoder layers as in examples/decoder_layer.py, a head kept in
8-bit integers (the layer that stands 4 bits least).  A step, captured in a CUDA
graph, is

    room for the tokens -> copy of shared pages -> embedding -> layers -> norm ->
    8-bit head -> penalties, temperature, choice of the token -> its history
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int4_group_quantized_int4g_gb300 as fl  # noqa: E402
from examples.decoder_layer import BLOCK, DecoderLayer  # noqa: E402


class Generator:
    """Layers, head and the books of one pool of pages.  Slot p * ways holds
    prompt p, the ways - 1 slots behind it its other continuations."""

    def __init__(self, prompts=4, ways=4, room=2048, layers=2, vocab=32000, pages=None, seed=0, **layer):
        self.prompts, self.ways, self.vocab = prompts, ways, vocab
        self.slots = prompts * ways
        self.layers = [DecoderLayer(batch=self.slots, room=room, seed=seed + i, **layer) for i in range(layers)]
        first = self.layers[0]
        self.device, hidden = first.device, first.hidden
        blocks = pages or first.cache[0].shape[0]
        # one set of books for all layers: their caches have the same pages
        self.refs = torch.zeros(blocks, dtype=torch.int32, device=self.device)
        self.table = torch.full((self.slots, -(-room // BLOCK)), -1, dtype=torch.int32, device=self.device)
        self.kv_lens = torch.zeros(self.slots, dtype=torch.int32, device=self.device)
        for one in self.layers:
            one.table = self.table
            one.cache = [c[:blocks].contiguous() for c in one.cache]
            one.scales = [c[:blocks].contiguous() for c in one.scales]
        g = torch.Generator(device=self.device)
        g.manual_seed(seed + 1000)
        self.embedding = torch.randn((vocab, hidden), generator=g, device=self.device).to(torch.bfloat16)
        self.norm_out = torch.ones(hidden, dtype=torch.bfloat16, device=self.device)
        self.head, self.head_scale = fl.fl_int8_quantize((torch.randn((vocab, hidden), generator=g, device=self.device)
                                                          * hidden ** -0.5).to(torch.bfloat16))
        # (all that a slot's table holds, and the token chosen behind them; rows of whole 16 bytes)
        self.history = torch.zeros((self.slots, self.table.shape[1] * BLOCK + 4), dtype=torch.int32, device=self.device)
        self.prompt_lens = torch.zeros(self.slots, dtype=torch.int32, device=self.device)
        # continuations differ in what a repeated token costs them, and in some tokens that each prefers
        way = torch.arange(self.slots, device=self.device) % ways
        liked = torch.randint(0, vocab, (self.slots, 50), generator=g, device=self.device, dtype=torch.int32)
        self.rules = dict(repetition=1 + 0.2 * way.float(), frequency=0.1 * way.float(), presence=0.05 * way.float(),
                          temperature=torch.full((self.slots,), 0.8, device=self.device),
                          bias_offsets=torch.arange(0, 50 * self.slots + 1, 50, dtype=torch.int32, device=self.device),
                          bias_ids=liked.view(-1), bias=torch.full((50 * self.slots,), 2.0, device=self.device))
        self.seqs = torch.arange(self.slots, dtype=torch.int32, device=self.device)
        self.token = torch.zeros(self.slots, dtype=torch.int32, device=self.device)

    def workspace(self, tokens):
        n = max(self.layers[0].workspace(tokens).numel(), fl.fl_int8_linear_workspace(self.slots, self.vocab, self.layers[0].hidden),
                fl.fl_logits_process_workspace(self.slots, self.vocab),
                fl.fl_kv8_pages_workspace(self.refs.numel(), *self.table.shape, BLOCK))
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    @property
    def pool(self):
        return self.refs, self.table, self.kv_lens

    def copy_pages(self, pairs, count, ws):
        one = self.layers
        fl.fl_kv8_pages_copy([x.cache[0] for x in one], [x.cache[1] for x in one], [x.scales[0] for x in one],
                             [x.scales[1] for x in one], pairs, count, status=ws)

    def layers_forward(self, tokens, positions, kv_lens, ws, keep=None, **seqs):
        """The stream after all layers, normed."""
        x = self.embedding.index_select(0, tokens)
        residual = torch.zeros_like(x)
        for i, one in enumerate(self.layers):
            x, residual = one.forward(x, residual, positions, kv_lens, ws, keep=keep[i] if keep else None, **seqs)
        return fl.fl_rmsnorm(x, self.norm_out, residual=residual)["y"]

    def choose(self, hidden, ws, moved=None, keep=None):
        """The next token of every slot, and its place in the history; slots that
        have not moved on (moved, truth values; None: all have) keep the one they have."""
        logits = fl.fl_int8_linear(hidden, self.head, self.head_scale, out_dtype=torch.float32, ws=ws)
        got = fl.fl_logits_process(logits, history=self.history, history_lens=self.kv_lens, prompt_lens=self.prompt_lens, **self.rules,
                                   ws=ws)
        if keep is not None:
            keep.update(hidden=hidden, logits=logits, history=self.history.clone(), history_lens=self.kv_lens.clone(), chosen=got)
        at = self.kv_lens.long()[:, None]
        token = got["token"]
        if moved is None:
            self.token.copy_(token)
        else:
            self.token.copy_(torch.where(moved, token, self.token))
            token = torch.where(moved, token, self.history.gather(1, at)[:, 0])
        self.history.scatter_(1, at, token[:, None])
        return got

    def start(self, prompts, ws):
        """prompts: a list of token lists.  Reads them and lets each have `ways` continuations."""
        if len(prompts) != self.prompts or not all(prompts):
            raise ValueError(f"expected {self.prompts} prompts of at least a token each")
        if min(map(min, prompts)) < 0 or max(map(max, prompts)) >= self.vocab:
            raise ValueError(f"a prompt's tokens are those of a vocabulary of {self.vocab}")
        dev = self.device
        lens = torch.zeros(self.slots, dtype=torch.int32)
        lens[::self.ways] = torch.tensor([len(p) for p in prompts], dtype=torch.int32)
        cu_q = torch.zeros(self.slots + 1, dtype=torch.int32)
        cu_q[1:] = lens.cumsum(0)
        cu_q, lens = cu_q.to(dev), lens.to(dev)
        flat = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=dev)
        firsts = self.seqs[::self.ways].contiguous()
        granted, pairs, count = fl.fl_kv8_pages_alloc(*self.pool, firsts, lens[::self.ways].contiguous(), BLOCK, ws=ws)
        if not bool(granted.all()):
            raise RuntimeError("the pool has too few pages for the prompts")
        positions = torch.cat([torch.arange(len(p), dtype=torch.int32) for p in prompts]).to(dev)
        hidden = self.layers_forward(flat, positions, self.kv_lens, ws, cu_q=cu_q, max_q=max(len(p) for p in prompts))
        if self.ways > 1:
            children = self.seqs.view(-1, self.ways)[:, 1:].contiguous()
            fl.fl_kv8_pages_fork(*self.pool, firsts[:, None].expand_as(children).contiguous(), children, BLOCK, status=ws)
        for i, p in enumerate(prompts):
            self.history[i * self.ways:(i + 1) * self.ways, :len(p)] = torch.tensor(p, dtype=torch.int32, device=dev)
        self.prompt_lens.copy_(self.kv_lens)
        last = (cu_q[1:][::self.ways] - 1).repeat_interleave(self.ways)
        return self.choose(hidden.index_select(0, last), ws)

    def step(self, new, ws, keep=None):
        """One token of every slot; new int32 [slots]: 1, or 0 for those that stay as
        they are.  A slot that gets no room (the pool is full, or its table) stays so
        too, and goes on with the token that it has when a later step finds room."""
        granted, pairs, count = fl.fl_kv8_pages_alloc(*self.pool, self.seqs, new, BLOCK, ws=ws)
        self.copy_pages(pairs, count, ws)
        # the others' rows are there, but of no token: nothing is written for them, and their
        # last tokens and the pages that they share stay
        moved = (granted > 0) & (new > 0)
        lens = self.kv_lens * moved
        positions = (lens - 1).clamp(min=0)
        steps = [{} for _ in self.layers] if keep is not None else None
        hidden = self.layers_forward(self.token.clamp(min=0), positions, lens, ws, keep=steps, max_q=1)
        if keep is not None:
            keep.update(granted=granted, pairs=pairs, count=count, layers=steps)
        return self.choose(hidden, ws, moved, keep)

    def end(self, slots, ws):
        """The sequences in these slots end; the pages in use move together."""
        fl.fl_kv8_pages_free(*self.pool, slots, BLOCK, status=ws)
        _, _, pairs, count, _ = fl.fl_kv8_pages_compact(*self.pool, BLOCK, status=ws)
        self.copy_pages(pairs, count, ws)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("prompts", 4), ("ways", 4), ("prompt", 500), ("steps", 64), ("layers", 4), ("vocab", 32000)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    gen = Generator(prompts=a.prompts, ways=a.ways, room=a.prompt + 2 * a.steps + 16, layers=a.layers, vocab=a.vocab)
    g = torch.Generator().manual_seed(0)
    prompts = [torch.randint(0, a.vocab, (a.prompt - 7 * i,), generator=g).tolist() for i in range(a.prompts)]
    ws = gen.workspace(a.prompt * a.prompts)
    gen.start(prompts, ws)
    held = int((gen.refs > 0).sum())
    print(f"{a.prompts} prompts, {gen.slots} continuations in {held} pages (without sharing {held * a.ways})")

    new = torch.ones(gen.slots, dtype=torch.int32, device=gen.device)
    step_ws = gen.workspace(gen.slots)
    gen.step(new, step_ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gen.step(new, step_ws)

    def run(steps):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(steps):
            graph.replay()
        end.record()
        end.synchronize()
        return 1e3 * start.elapsed_time(end) / steps

    print(f"{a.steps} steps of {gen.slots} tokens: {run(a.steps):.0f} us a step, {int((gen.refs > 0).sum())} pages")
    ended = gen.seqs.view(-1, a.ways)[:, a.ways // 2:].contiguous()   # half of the continuations end
    new.view(-1, a.ways)[:, a.ways // 2:] = 0
    gen.end(ended, ws)
    print(f"half of them ended: {int((gen.refs > 0).sum())} pages; {run(a.steps):.0f} us a step")
    status = fl.fl_int4g_status(ws) or fl.fl_int4g_status(step_ws)
    print(f"two continuations: {gen.history[:2, a.prompt:a.prompt + 8].tolist()}; status {fl.fl_strerror(status)}")


if __name__ == "__main__":
    main()
