"""The serving operators and the example around them at the edges of their use, on
the GPU: threads on one stream, pools that are full, sums past 2^24."""
import threading

import numpy as np
import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from examples.generate import BLOCK, Generator
from oracle import serving_oracle as O
from test_gpu_generate import _books, _check_step, _values

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int4_group_quantized_int4g_gb300 import _build
    _build.build()
    fl.lib()


@pytest.mark.parametrize("captured", [False, True])
def test_continuations_without_room_wait_for_it(captured):
    """A prompt of 70 tokens, three continuations and a pool of three pages: one copies
    the last page, the others get no room until it ends."""
    gen = Generator(prompts=1, ways=3, room=192, layers=2, vocab=500, pages=3, hidden=128, heads=2, kv_heads=1, dim=64, experts=2,
                    inter=128, top_k=1)
    pool = O.Pool(3, 3, gen.table.shape[1], BLOCK)
    ws = gen.workspace(70)
    gen.start([list(range(70))], ws)
    pool.alloc([0], [70])
    pool.fork([0, 0], [1, 2])
    _books(gen, pool)
    new = torch.ones(3, dtype=torch.int32, device=DEV)
    keep = {}
    if captured:
        gen.step(torch.zeros_like(new), ws)          # (first calls of every kernel; nobody moves)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            gen.step(new, ws, keep)

    def step(values):
        new.copy_(torch.tensor(values, dtype=torch.int32))
        if captured:
            graph.replay()
        else:
            gen.step(new, ws, keep)
        granted, pairs = pool.alloc([0, 1, 2], values)
        assert keep["granted"].tolist() == granted and int(keep["count"]) == len(pairs)
        _books(gen, pool)
        return granted
    held = [[_values(gen, i, s) for i in range(2)] for s in range(3)]
    token, history = gen.token.clone(), gen.history.clone()
    for _ in range(2):
        assert step([1, 1, 1]) == [1, 0, 0]
        _check_step(gen, keep, (0,))
        for s in (1, 2):
            assert all(np.array_equal(_values(gen, i, s), held[s][i]) for i in range(2))
        assert torch.equal(gen.token[1:], token[1:]) and torch.equal(gen.history[1:], history[1:])
    # (tokens of the page that is written next may be rounded again)
    assert all(np.array_equal(_values(gen, i, 0)[:, :, :64], held[0][i][:, :, :64]) for i in range(2))
    gen.end(torch.tensor([0], dtype=torch.int32, device=DEV), ws)
    pool.free([0])
    pool.compact()
    for _ in range(2):
        assert step([0, 1, 1])[1:] == [1, 1]
        _check_step(gen, keep, (1, 2))
    assert gen.kv_lens.tolist() == [0, 72, 72]
    assert torch.equal(gen.history[1:, 70], token[1:])
    assert all(np.array_equal(_values(gen, i, s)[:, :, :64], held[s][i][:, :, :64]) for i in range(2) for s in (1, 2))
    assert fl.fl_int4g_status(ws) == 0


# ------------------------------------------------------------------ linear

def _in_batches(x, w, t):
    """The first row's product, alone and in batches whose sums are divided otherwise."""
    return [fl.fl_int8_linear(x[:M], w, t, out_dtype=torch.float32)[0].double().cpu().numpy() for M in (1, 8, 16, 17, 64, 300, 1000)]


def test_a_row_is_the_same_in_every_batch_while_sums_are_below_2_24():
    """1040 products of 127 and 127, of one sign: 16.774e6 of 2^24 = 16.777e6."""
    x = torch.full((1000, 1040), 3.0, dtype=torch.bfloat16, device=DEV)
    w = torch.full((300, 1040), 127, dtype=torch.int8, device=DEV)
    w[1::2] = -127
    w[5] = torch.arange(1040, device=DEV) % 255 - 127
    t = torch.linspace(0.5, 2.0, 300, device=DEV) * 1e-3
    got = _in_batches(x, w, t)
    assert all(np.array_equal(g, got[0]) for g in got)


@pytest.mark.parametrize("K", [8192, 16384])
def test_a_row_in_batches_past_2_24(K):
    """Sums of 15e6, below 2^24, and of 30e6.  Past 2^24 a sum is rounded, where
    depends on the batch: each of the K / 16 steps and of joining the parts by at
    most a step, 2^-23 of it, on either side, and both results by three roundings to
    fp32 more."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy(np.abs(rng.standard_normal((1000, K))).astype(np.float32)).to(torch.bfloat16).to(DEV)
    w = torch.from_numpy(rng.integers(0, 128, (300, K)).astype(np.int8)).to(DEV)
    t = torch.from_numpy((np.exp(0.3 * rng.standard_normal(300)) * 1e-3).astype(np.float32)).to(DEV)
    q, s = O.quantize8(x[:1].double().cpu().numpy())
    dot, scale = O.linear8(q, s, w.cpu().numpy(), t.double().cpu().numpy())
    assert dot.max() < 2 ** 24 if K == 8192 else dot.min() > 2 ** 24
    ref = (dot * scale)[0]
    step = ref * ((K / 16 + 20) * 2.0 ** -23 + 3 * 2.0 ** -24)
    got = _in_batches(x, w, t)
    for g, again in zip(got, _in_batches(x, w, t)):
        assert np.array_equal(g, again) and (K == 16384 or np.array_equal(g, got[0]))
        assert np.all(np.abs(g - ref) <= step) and np.all(np.abs(g - got[0]) <= 2 * step)


# ----------------------------------------------------------------- threads

def test_threads_on_one_stream():
    """Calls of several launches from four threads at once, without workspaces of the
    callers', give what they give one after another."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    w = torch.randint(-127, 128, (1000, 512), generator=g, device=DEV, dtype=torch.int8)
    t = torch.rand(1000, generator=g, device=DEV)
    xs = [torch.randn((m, 512), generator=g, device=DEV).to(torch.bfloat16) for m in (1, 9, 40, 150)]
    rows = [torch.randn((m, 20011), generator=g, device=DEV) for m in (1, 5, 300, 600)]

    def both(i):
        got = fl.fl_logits_process(rows[i])
        return [fl.fl_int8_linear(xs[i], w, t), got["logits"], got["token"], got["lse"]]
    want = [both(i) for i in range(4)]
    torch.cuda.synchronize()
    barrier = threading.Barrier(4)
    same, errors = [True] * 4, []

    def run(i):
        try:
            torch.cuda.set_device(DEV)
            barrier.wait()
            for _ in range(100):
                same[i] &= all(torch.equal(a, b) for a, b in zip(both(i), want[i]))
        except Exception as e:       # noqa: BLE001 (told by the test)
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and all(same)
