"""The decoder layer of examples/decoder_layer.py: every step of a prompt and of
a captured token step against the float64 oracles, on the step's own inputs."""
import os
import sys

import numpy as np
import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from oracle import int4g_oracle as W
from oracle import layer_oracle as O

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from decoder_layer import DecoderLayer  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int4_group_quantized_int4g_gb300 import _build
    _build.build()
    fl.lib()


def _np(t):
    return t.detach().double().cpu().numpy()


def _triple(t):
    return t[0].cpu().numpy(), t[1].cpu().numpy().view(np.uint16), t[2].cpu().numpy()


def _near(got, ref, tol, what):
    err = np.abs(_np(got) - ref)
    assert np.all(err <= tol), (what, np.max(err - tol))


def _check(layer, x, residual, positions, kv_lens, cu_q, k, y, out_res, cache):
    """k: the kept steps; cache: copies of the codes and scales before the call."""
    half, slack = 2.0 ** -8, 2.0 ** -18          # half a step of bf16; fp32 arithmetic
    hq, hk, d = layer.heads, layer.kv_heads, layer.dim
    s, n = O.rmsnorm(_np(x), _np(residual), _np(layer.norm_in), 1e-6)
    _near(k["norm_in"], n, (half + slack) * np.abs(n), "norm")
    _near(k["residual_in"], s, (half + slack) * np.abs(s), "residual")
    xf = _np(k["norm_in"])
    qkv = _triple(layer.triples["qkv"])
    _near(k["qkv"].reshape(len(xf), -1), W.linear(xf, *qkv), W.linear_tolerance(xf, *qkv), "qkv")
    axis = [0] * (d // 2)
    raw = _np(k["qkv"])
    for name, part, gain in (("q", raw[:, :hq], layer.norm_q), ("k", raw[:, hq:hq + hk], layer.norm_k)):
        normed = O.rmsnorm(part, None, _np(gain), 1e-6)[1]
        ref = O.rope(normed, positions[None], _np(layer.inv_freq), axis, True)
        both = np.abs(normed[..., :d // 2]) + np.abs(normed[..., d // 2:])
        # the norm's rounding turns with the pair, then the result's own
        _near(k[name], ref, half * np.abs(ref) + (half + 1e-5) * np.concatenate([both, both], -1), name)
    codes, scales = cache
    for i, name in enumerate("kv"):
        O.append(_np(k[name]), codes[i], scales[i], _np(layer.table).astype(int), kv_lens, cu_q, layer.fmt)
        assert np.array_equal(layer.cache[i].cpu().numpy(), codes[i]) and np.array_equal(layer.scales[i].cpu().numpy(), scales[i])
    ref, _, tol, _ = O.attention(_np(k["q"]), codes[0], codes[1], scales[0], scales[1], _np(layer.table).astype(int), kv_lens,
                                 cu_q, layer.fmt, d ** -0.5)
    _near(k["attention"], ref, tol, "attention")
    af, o = _np(k["attention"]).reshape(len(xf), -1), _triple(layer.triples["o"])
    _near(k["o"], W.linear(af, *o), W.linear_tolerance(af, *o), "o")
    s, n = O.rmsnorm(_np(k["o"]), _np(k["residual_in"]), _np(layer.norm_post), 1e-6)
    _near(k["norm_post"], n, (half + slack) * np.abs(n), "second norm")
    _near(out_res, s, (half + slack) * np.abs(s), "second residual")
    w13 = [_triple(layer.triples[("w13", e)]) for e in range(layer.experts)]
    w2 = [_triple(layer.triples[("w2", e)]) for e in range(layer.experts)]
    ref, tol, _, _ = W.moe(_np(k["norm_post"]), k["logits"].cpu().numpy(), layer.top_k, w13, w2, W.SOFTMAX, True)
    _near(y, ref, tol, "experts")


@pytest.mark.parametrize("fmt", [fl.FL_KV8_E4M3, fl.FL_KV8_INT8])
@pytest.mark.parametrize("lens", [[70, 1, 33], [5, 200, 129]])
def test_decoder_layer(fmt, lens):
    layer = DecoderLayer(hidden=256, heads=6, kv_heads=2, dim=64, experts=4, inter=128, top_k=2, batch=3, room=256, fmt=fmt)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def rows(n):
        return [torch.randn((n, 256), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]

    def host():
        return [c.cpu().numpy().copy() for c in layer.cache], [c.cpu().numpy().copy() for c in layer.scales]

    # the prompts in one ragged call
    T, cu = sum(lens), [0, *np.cumsum(lens).tolist()]
    ws = layer.workspace(T)
    x, res = rows(T)
    pos = np.concatenate([np.arange(n) for n in lens])
    keep, cache = {}, host()
    y, out = layer.forward(x, res, torch.tensor(pos, dtype=torch.int32, device=DEV),
                           torch.tensor(lens, dtype=torch.int32, device=DEV), ws,
                           cu_q=torch.tensor(cu, dtype=torch.int32, device=DEV), max_q=max(lens), keep=keep)
    _check(layer, x, res, pos, lens, cu, keep, y, out, cache)

    # two tokens for each sequence by one captured step
    x, res = rows(3)
    p, n = torch.tensor(lens, dtype=torch.int32, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV) + 1
    step_ws = layer.workspace(3)
    keep, graph = {}, torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y, out = layer.forward(x, res, p, n, step_ws, max_q=1, keep=keep)
    for i in range(2):
        if i:
            for t, new in zip((x, res), rows(3)):
                t.copy_(new)
            p.add_(1)
            n.add_(1)
        cache = host()
        graph.replay()
        torch.cuda.synchronize()
        _check(layer, x, res, np.array(lens) + i, [v + 1 + i for v in lens], [0, 1, 2, 3], keep, y, out, cache)
    assert fl.fl_int4g_status(ws) == 0 and fl.fl_int4g_status(step_ws) == 0
