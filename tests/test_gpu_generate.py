"""Several continuations of each prompt (examples/generate.py): pages, cache,
attention, the 8-bit head and the choice of a token together, step by step
against the float64 oracles on each step's own inputs, captured steps too."""
import os
import sys

import numpy as np
import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from oracle import layer_oracle as LO
from oracle import serving_oracle as O

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.generate import BLOCK, Generator  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int4_group_quantized_int4g_gb300 import _build
    _build.build()
    fl.lib()


def _np(t):
    return t.detach().double().cpu().numpy()


def _books(gen, pool):
    refs, table, lens = (t.cpu().tolist() for t in gen.pool)
    assert refs == pool.refs and lens == pool.lens
    for s, n in enumerate(lens):
        assert table[s][:pool.pages(n)] == pool.table[s][:pool.pages(n)]


def _values(gen, layer, slot):
    """Keys and values that a slot's tokens have in the cache, [2, heads, tokens, dim]."""
    one, n = gen.layers[layer], int(gen.kv_lens[slot])
    row = gen.table[slot].cpu().numpy()
    return np.stack([LO.gather(one.cache[i].cpu().numpy(), _np(one.scales[i]), row, n, one.fmt) for i in range(2)])


def _check_step(gen, keep, live):
    lens = gen.kv_lens.cpu().numpy()
    cu = np.arange(gen.slots + 1)
    for one, k in zip(gen.layers, keep["layers"]):
        cache = [c.cpu().numpy() for c in one.cache]
        out, _, tol, _ = LO.attention(_np(k["q"]), cache[0], cache[1], _np(one.scales[0]), _np(one.scales[1]),
                                      gen.table.cpu().numpy(), lens, cu, one.fmt, one.dim ** -0.5)
        for s in live:
            assert np.all(np.abs(_np(k["attention"])[s] - out[s]) <= tol[s]), s
    # the head: sums of whole numbers below 2^24 are exact, two roundings of fp32 behind them
    q, scale = O.quantize8(_np(keep["hidden"]))
    dot, both = O.linear8(q, scale, gen.head.cpu().numpy(), _np(gen.head_scale))
    logits = keep["logits"].cpu().numpy()
    assert np.abs(dot).max() < 2 ** 24
    assert np.all(np.abs(logits - dot * both) <= 3 * 2.0 ** -24 * np.abs(dot * both) + 1e-44)
    rules = {k: v.cpu().numpy() for k, v in gen.rules.items()}
    want, token, lse, logprob = O.logits(logits, history=keep["history"].cpu().numpy(), history_lens=keep["history_lens"].cpu().numpy(),
                                         prompt_lens=gen.prompt_lens.cpu().numpy(), **rules, real=np.float32)
    got = keep["chosen"]
    assert np.array_equal(got["logits"].cpu().numpy(), want) and np.array_equal(got["token"].cpu().numpy(), token)
    # (the bound of lse and logprob is derived in test_gpu_serving_ops.py)
    for name, ref in (("lse", lse), ("logprob", logprob)):
        assert np.all(np.abs(_np(got[name]) - ref) <= 2.0 ** -18 + 2.0 ** -22 * (np.abs(ref) + np.abs(lse)))
    for s in live:
        assert int(gen.history[s, lens[s]]) == token[s]


@pytest.mark.parametrize("lengths", [(70, 131), (64, 1)])
def test_continuations_of_shared_prompts(lengths):
    gen = Generator(prompts=2, ways=3, room=256, layers=2, vocab=1003, pages=21, hidden=256, heads=4, kv_heads=2, dim=64, experts=4,
                    inter=128, top_k=2)
    pool = O.Pool(21, 6, gen.table.shape[1], BLOCK)
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, 1003, n).tolist() for n in lengths]
    ws = gen.workspace(sum(lengths))
    gen.start(prompts, ws)
    pool.alloc([0, 3], list(lengths))
    pool.fork([0, 0, 3, 3], [1, 2, 4, 5])
    _books(gen, pool)
    assert sum(r > 0 for r in pool.refs) == sum(-(-n // BLOCK) for n in lengths)      # shared, whatever the ways
    full = [n // BLOCK * BLOCK for n in lengths]                                      # tokens of whole pages: never written again
    before = [[_values(gen, i, 3 * p)[:, :, :full[p]] for p in range(2)] for i in range(2)]

    new = torch.ones(6, dtype=torch.int32, device=DEV)
    for step in range(5):
        keep = {}
        gen.step(new, ws, keep)
        granted, pairs = pool.alloc(list(range(6)), [1] * 6)
        assert keep["granted"].tolist() == granted == [1] * 6 and int(keep["count"]) == len(pairs)
        assert len(pairs) == (sum(2 for n in lengths if n % BLOCK) if step == 0 else 0)
        _books(gen, pool)
        _check_step(gen, keep, range(6))
    # nobody has written into the prompt's whole pages
    for i in range(2):
        for s in range(6):
            assert np.array_equal(_values(gen, i, s)[:, :, :full[s // 3]], before[i][s // 3])

    # the prompts' own sequences end; what is left moves together and goes on
    held = {s: [_values(gen, i, s) for i in range(2)] for s in (1, 2, 4, 5)}
    gen.end(torch.tensor([0, 3], dtype=torch.int32, device=DEV), ws)
    pool.free([0, 3])
    pool.compact()
    _books(gen, pool)
    live = sum(r > 0 for r in pool.refs)
    assert not any(pool.refs[live:])
    for s, want in held.items():
        assert all(np.array_equal(_values(gen, i, s), want[i]) for i in range(2))
    new[0], new[3] = 0, 0
    keep = {}
    gen.step(new, ws, keep)
    pool.alloc(list(range(6)), [0, 1, 1, 0, 1, 1])
    _books(gen, pool)
    _check_step(gen, keep, (1, 2, 4, 5))
    assert fl.fl_int4g_status(ws) == 0


def test_captured_steps_are_the_same_as_others():
    def make():
        gen = Generator(prompts=1, ways=4, room=192, layers=1, vocab=500, hidden=128, heads=2, kv_heads=1, dim=64, experts=2, inter=128,
                        top_k=1)
        ws = gen.workspace(40)
        gen.start([list(range(40))], ws)
        return gen, ws
    new = torch.ones(4, dtype=torch.int32, device=DEV)
    a, ws_a = make()
    for _ in range(60):                      # across the ends of pages
        a.step(new, ws_a)
    b, ws_b = make()
    b.step(new, ws_b)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.step(new, ws_b)
    for _ in range(59):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.history, b.history) and torch.equal(a.kv_lens, b.kv_lens) and torch.equal(a.refs, b.refs)
    assert all(torch.equal(x, y) for x, y in zip(a.layers[0].cache, b.layers[0].cache))
    assert fl.fl_int4g_status(ws_a) == 0 and fl.fl_int4g_status(ws_b) == 0
