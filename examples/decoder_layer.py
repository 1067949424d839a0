"""A decoder layer of int4g weights, end to end through this library: a prompt,
then tokens one by one, captured in a CUDA graph.

    python examples/decoder_layer.py [--prompt 2000] [--steps 32] [--batch 4] [--format e4m3|int8]

Random weights of a Qwen3-MoE-shaped layer (hidden 2048, 32 query and 4 key
heads of 128, 128 experts of 768, top-8).  Every step of the layer is one of the
library's calls:

    norm + residual -> int4g QKV -> norm of each query and key head -> rotary
    positions -> write into the 8-bit cache -> attention over the cache ->
    int4g output -> norm + residual -> router -> int4g experts
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int4_group_quantized_int4g_gb300 as fl  # noqa: E402

BLOCK = 64   # tokens of a cache block


class DecoderLayer:
    """Weights, cache and workspace of one layer for a batch of sequences."""

    def __init__(self, hidden=2048, heads=32, kv_heads=4, dim=128, experts=128, inter=768, top_k=8, batch=4, room=4096,
                 fmt=fl.FL_KV8_E4M3, base=1e6, seed=0, device="cuda"):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        self.experts, self.inter, self.top_k, self.batch, self.fmt = experts, inter, top_k, batch, fmt
        self.device = torch.device(device)
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.triples = {}

        def weight(name, rows, cols):   # interleaved int4g weights of a random matrix
            t = fl.fl_int4g_quantize(torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5)
            self.triples[name] = t
            return fl.fl_int4g_repack(*t, rows, cols)

        def gain(n):
            return (1 + 0.1 * torch.randn(n, generator=g, device=device)).to(torch.bfloat16)

        self.w_qkv = weight("qkv", (heads + 2 * kv_heads) * dim, hidden)
        self.w_o = weight("o", hidden, heads * dim)
        self.w13 = torch.cat([weight(("w13", e), 2 * inter, hidden) for e in range(experts)])
        self.w2 = torch.cat([weight(("w2", e), hidden, inter) for e in range(experts)])
        self.w_router = (torch.randn((experts, hidden), generator=g, device=device) * hidden ** -0.5).to(torch.bfloat16)
        self.norm_in, self.norm_post = gain(hidden), gain(hidden)
        self.norm_q, self.norm_k = gain(dim), gain(dim)
        self.inv_freq = (base ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2))).to(device)
        # the cache: every sequence gets the blocks for `room` tokens, in a shuffled order
        per = -(-room // BLOCK)
        blocks = batch * per
        self.cache = [torch.zeros((blocks, kv_heads, BLOCK, dim), dtype=torch.uint8, device=device) for _ in range(2)]
        self.scales = [torch.ones((blocks, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
        self.table = torch.randperm(blocks, generator=g, device=device).to(torch.int32).view(batch, per)

    def workspace(self, tokens):
        """One zero-filled workspace for all calls on up to `tokens` tokens."""
        n = max(fl.fl_int4g_linear_workspace(tokens, self.w_rows("qkv"), self.hidden),
                fl.fl_int4g_linear_workspace(tokens, self.hidden, self.heads * self.dim),
                fl.fl_kv8_attention_workspace(tokens, self.batch, self.heads, self.kv_heads, self.dim),
                fl.fl_moe_router_logits_workspace(tokens, self.hidden, self.experts),
                fl.fl_moe_int4g_workspace(tokens, self.experts, self.top_k, self.hidden, self.inter, False))
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    def w_rows(self, name):
        return self.triples[name][0].shape[0]

    def forward(self, x, residual, positions, kv_lens, ws, cu_q=None, max_q=None, keep=None):
        """x: what the layer before added to the residual stream, residual: the
        stream before it (both bf16 [T, hidden]); positions int32 [T], kv_lens
        int32 [batch] with the new tokens.  Returns (what this layer adds,
        the stream before it).  keep: a dict that gets the steps' results."""
        T, hq, hk, d = x.shape[0], self.heads, self.kv_heads, self.dim
        n = fl.fl_rmsnorm(x, self.norm_in, residual=residual)
        qkv = fl.fl_int4g_linear(n["y"], self.w_qkv, self.w_rows("qkv"), ws=ws).view(T, hq + 2 * hk, d)
        if keep is not None:
            keep.update(norm_in=n["y"], residual_in=n["residual"], qkv=qkv.clone())
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        fl.fl_rmsnorm(q, self.norm_q, y=q)
        fl.fl_rmsnorm(k, self.norm_k, y=k)
        fl.fl_rope(q, k, positions, self.inv_freq, q_out=q, k_out=k)
        seqs = dict(cu_q=cu_q, max_q=max_q, fmt=self.fmt)
        fl.fl_kv8_append(k, v, *self.cache, *self.scales, self.table, kv_lens, status=ws, **seqs)
        a = fl.fl_kv8_attention(q, *self.cache, *self.scales, self.table, kv_lens, ws=ws, **seqs)
        o = fl.fl_int4g_linear(a.view(T, hq * d), self.w_o, self.hidden, ws=ws)
        m = fl.fl_rmsnorm(o, self.norm_post, residual=n["residual"])
        logits = fl.fl_moe_router_logits(m["y"], self.w_router, ws=ws)
        y = fl.fl_moe_int4g(m["y"], logits, self.top_k, self.inter, self.w13, self.w2, ws=ws)
        if keep is not None:
            keep.update(q=q, k=k, v=v, attention=a, o=o, norm_post=m["y"], residual_post=m["residual"], logits=logits)
        return y, m["residual"]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompt", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--format", choices=("e4m3", "int8"), default="e4m3")
    a = ap.parse_args()
    dev = "cuda"
    layer = DecoderLayer(batch=a.batch, room=a.prompt + a.steps + 8,
                         fmt=fl.FL_KV8_E4M3 if a.format == "e4m3" else fl.FL_KV8_INT8)

    def timed(run):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        run()
        end.record()
        end.synchronize()
        return start.elapsed_time(end)

    # prompts, in parts that the expert layer takes at once (tokens x top-k <= 16384)
    part = min(a.prompt, 16384 // layer.top_k // a.batch)
    ws = layer.workspace(part * a.batch)
    ms = done = 0
    while done < a.prompt:
        n = min(part, a.prompt - done)
        x = torch.randn((a.batch * n, layer.hidden), device=dev).to(torch.bfloat16)
        pos = torch.arange(done, done + n, dtype=torch.int32, device=dev).repeat(a.batch)
        lens = torch.full((a.batch,), done + n, dtype=torch.int32, device=dev)
        ms += timed(lambda: layer.forward(x, torch.zeros_like(x), pos, lens, ws, max_q=n))
        done += n
    print(f"prompt: {a.batch} x {a.prompt} tokens in {ms:.2f} ms a layer")

    # tokens one by one: one captured step, its lengths and positions moved on in place
    x = torch.randn((a.batch, layer.hidden), device=dev).to(torch.bfloat16)
    res = torch.zeros_like(x)
    pos = torch.full((a.batch,), a.prompt, dtype=torch.int32, device=dev)
    lens = pos + 1
    step_ws = layer.workspace(a.batch)
    layer.forward(x, res, pos, lens, step_ws, max_q=1)   # (first calls of every kernel)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.forward(x, res, pos, lens, step_ws, max_q=1)
        pos.add_(1)
        lens.add_(1)
    graph.replay()
    ms = timed(lambda: [graph.replay() for _ in range(a.steps)])
    status = fl.fl_int4g_status(step_ws) or fl.fl_int4g_status(ws)
    print(f"tokens: {a.steps} steps of {a.batch}, {1e3 * ms / a.steps:.1f} us a layer and step; status {fl.fl_strerror(status)}")


if __name__ == "__main__":
    main()
