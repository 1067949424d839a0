"""Host side of the serving operators at the edges of their use: several threads,
tensors of other devices, outputs over inputs, pools that are full.  No GPU."""
import ctypes
import threading
import types
import weakref

import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from examples import generate
from int4_group_quantized_int4g_gb300 import _build
from oracle import serving_oracle as O


# ------------------------------------------------------------ workspaces

class Buffer:
    def __init__(self, n):
        self.n = n

    def numel(self):
        return self.n

    def data_ptr(self):
        return id(self)


def _fake_torch(state):
    """What the binding's workspaces need of torch, on a stream of the handle 77."""
    return types.SimpleNamespace(zeros=lambda n, **kw: Buffer(n), uint8=torch.uint8,
                                 _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: 77),
                                 cuda=types.SimpleNamespace(is_current_stream_capturing=lambda: state["capturing"]))


def test_threads_on_one_stream_have_workspaces_of_their_own(monkeypatch):
    """A call of several launches hands its codes over in the workspace; the
    launches of two threads on one stream come in any order."""
    monkeypatch.setattr(fl, "_torch", lambda: _fake_torch({"capturing": False}))
    monkeypatch.setattr(fl, "_WS", {})
    monkeypatch.setattr(fl, "_OUTGROWN", [])
    dev = torch.device("cuda", 0)
    barrier = threading.Barrier(3)
    got = {}

    def calls(i):
        barrier.wait()
        got[i] = [fl._space(None, 4000, dev, 77)[0], fl._workspace(3000, dev), fl._space(None, 9000, dev, 77)[0], fl._workspace(9000, dev)]
        barrier.wait()          # (all threads live at once)
    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    barrier.wait()
    barrier.wait()
    for t in threads:
        t.join()
    assert all(a is not b for a in got[0] for b in got[1])
    for mine in got.values():                              # one of each thread's, grown on demand
        assert mine[0] is mine[1] and mine[2] is mine[3] and mine[2].numel() >= 9000
    mine = fl._workspace(9000, dev)
    assert fl._space(None, 9000, dev, 77)[0] is mine and fl._workspace(100, dev) is mine


# ------------------------------------------------------------- generation

def _generator(monkeypatch, blocks, lens, ways):
    """examples/generate.py's books and steps on the CPU, the library's calls replaced by
    the oracle's pool and a layer that notes which token each place of the cache holds."""
    pool = O.Pool(blocks, len(lens) * ways, 2, generate.BLOCK)
    cache = {}

    def to_tensors(gen):
        gen.refs.copy_(torch.tensor(pool.refs)), gen.kv_lens.copy_(torch.tensor(pool.lens)), gen.table.copy_(torch.tensor(pool.table))

    def alloc(refs, table, kv_lens, seqs, new, block, ws=None):
        granted, pairs = pool.alloc(seqs.tolist(), new.tolist())
        to_tensors(gen)
        flat = pairs + [(-1, -1)] * (len(granted) - len(pairs))
        return (torch.tensor(granted, dtype=torch.int32), torch.tensor(flat, dtype=torch.int32),
                torch.tensor([len(pairs)], dtype=torch.int32))

    def copy(k, v, a, b, pairs, count, status=None):
        for f, t in pairs[:int(count)].tolist():
            for off in range(generate.BLOCK):
                cache.pop((t, off), None)
                if (f, off) in cache:
                    cache[t, off] = cache[f, off]

    class Layer:
        cache, scales = [None, None], [None, None]

        def forward(self, x, residual, positions, kv_lens, ws, keep=None, max_q=None, **seqs):
            for s, n in enumerate(kv_lens.tolist()):     # a row a slot, the last of its tokens; none of an empty one
                if n:
                    place = (pool.table[s][(n - 1) // generate.BLOCK], (n - 1) % generate.BLOCK)
                    assert pool.refs[place[0]] == 1, "written into a shared page"
                    cache[place] = (s, n - 1, int(gen.token[s]))
            return x, residual
    gen = object.__new__(generate.Generator)
    slots = len(lens) * ways
    gen.prompts, gen.ways, gen.vocab, gen.slots, gen.layers, gen.device = len(lens), ways, 50, slots, [Layer()], torch.device("cpu")
    gen.refs, gen.table = torch.zeros(blocks, dtype=torch.int32), torch.full((slots, 2), -1, dtype=torch.int32)
    gen.kv_lens, gen.token = torch.zeros(slots, dtype=torch.int32), torch.arange(30, 30 + slots, dtype=torch.int32)
    gen.embedding, gen.norm_out, gen.head, gen.head_scale, gen.rules = torch.zeros((50, 8)), None, None, None, {}
    gen.history = torch.zeros((slots, 2 * generate.BLOCK + 4), dtype=torch.int32)
    gen.prompt_lens, gen.seqs = torch.zeros(slots, dtype=torch.int32), torch.arange(slots, dtype=torch.int32)
    calls = [0]

    def process(logits, **kw):
        calls[0] += 1
        return {"token": torch.arange(slots, dtype=torch.int32) + 10 * calls[0] % 40}
    stub = types.SimpleNamespace(fl_kv8_pages_alloc=alloc, fl_kv8_pages_copy=copy, fl_logits_process=process,
                                 fl_rmsnorm=lambda x, w, residual=None: {"y": x}, fl_int8_linear=lambda x, *a, **kw: x)
    monkeypatch.setattr(generate, "fl", stub)
    firsts = list(range(0, slots, ways))
    pool.alloc(firsts, list(lens))
    for s, n in zip(firsts, lens):
        for j in range(n):
            cache[pool.table[s][j // generate.BLOCK], j % generate.BLOCK] = ("prompt", j, 0)
        children = [s + i for i in range(1, ways)]
        pool.fork([s] * len(children), children)
        for c in [s] + children:
            gen.history[c, n] = gen.token[c]
    to_tensors(gen)
    return gen, pool, cache, lambda: to_tensors(gen)


def test_a_slot_without_room_stays_as_it_is(monkeypatch):
    """Three continuations of 20 tokens and one page left: the first copies, the others
    get no room, write nothing and keep their tokens until the first one ends."""
    gen, pool, cache, sync = _generator(monkeypatch, 2, (20,), 3)
    new = torch.ones(3, dtype=torch.int32)
    before, tokens, history = dict(cache), gen.token.clone(), gen.history.clone()
    keep = {}
    gen.step(new, None, keep)
    assert keep["granted"].tolist() == [1, 0, 0] and gen.kv_lens.tolist() == [21, 20, 20]
    assert {k: v for k, v in cache.items() if k[0] == 0} == before                    # the prompt's page
    assert cache[1, 20] == (0, 20, 30)
    assert torch.equal(gen.token[1:], tokens[1:]) and torch.equal(gen.history[1:], history[1:])
    assert int(gen.history[0, 21]) == int(gen.token[0]) == 10
    pool.free([0])
    sync()
    gen.step(torch.tensor([0, 1, 1], dtype=torch.int32), None, keep)
    assert keep["granted"].tolist() == [1, 1, 1] and gen.kv_lens.tolist() == [0, 21, 21]
    assert cache[1, 20] == (1, 20, 31) and cache[0, 20] == (2, 20, 32)
    assert gen.history[1:, 20].tolist() == [31, 32] and torch.equal(gen.history[1:, 21], gen.token[1:])


def test_a_live_slot_that_takes_no_token_stays_as_it_is(monkeypatch):
    gen, pool, cache, _ = _generator(monkeypatch, 6, (20, 64), 2)
    before, tokens, history = dict(cache), gen.token.clone(), gen.history.clone()
    gen.step(torch.tensor([0, 1, 0, 0], dtype=torch.int32), None)
    assert {k: v for k, v in cache.items() if k in before} == before and len(cache) == len(before) + 21
    still = [0, 2, 3]
    assert torch.equal(gen.token[still], tokens[still]) and torch.equal(gen.history[still], history[still])
    assert gen.kv_lens.tolist() == [20, 21, 64, 64]


def test_the_last_token_of_a_full_table_has_a_place(monkeypatch):
    """A slot may fill its table's last page; the token chosen then stands behind its
    tokens, not over the last one."""
    made = {}

    class Layer:
        hidden, device = 8, torch.device("cpu")

        def __init__(self, batch, room, seed, **kw):
            per = -(-room // generate.BLOCK)
            self.cache = [torch.zeros((batch * per, 1, 1, 1), dtype=torch.uint8) for _ in range(2)]
            self.scales = [torch.zeros((batch * per, 1)) for _ in range(2)]
    monkeypatch.setattr(generate, "DecoderLayer", Layer)
    monkeypatch.setattr(generate, "fl", types.SimpleNamespace(
        fl_int8_quantize=lambda x: (x, x), fl_int8_linear=lambda x, *a, **kw: x,
        fl_logits_process=lambda x, **kw: made.update(kw) or {"token": torch.full((2,), 7, dtype=torch.int32)}))
    for room in (100, 128):
        gen = generate.Generator(prompts=1, ways=2, room=room, layers=1, vocab=20)
        full = gen.table.shape[1] * generate.BLOCK
        gen.history.fill_(3)
        gen.kv_lens.copy_(torch.tensor([full, room]))
        gen.choose(torch.zeros((2, 8)), None)
        assert gen.history[0, :full].tolist() == [3] * full and int(gen.history[0, full]) == 7
        assert gen.history[1, :room].tolist() == [3] * room and int(gen.history[1, room]) == 7
        assert made["history"].stride(0) % 4 == 0          # (rows of whole 16 bytes)


@pytest.mark.parametrize("prompts", [[[1, 2], []], [[], [1]], [[1, 2]], [[1], [2], [3]], [[1, 50], [2]], [[1], [-1]]])
def test_prompts_that_cannot_be_read_are_refused(monkeypatch, prompts):
    """None, too few or too many, or tokens outside the vocabulary, before any call: an
    empty one has no last token to go on from, and others are read as indices."""
    gen, pool, cache, _ = _generator(monkeypatch, 6, (20, 64), 2)
    books = [t.clone() for t in gen.pool]
    with pytest.raises(ValueError):
        gen.start(prompts, None)
    assert all(torch.equal(a, b) for a, b in zip(gen.pool, books))


# ------------------------------------------------- outputs over inputs

@pytest.fixture(scope="module")
def L():
    _build.build()
    return fl.lib()


def _runs(rc):
    """Right as far as overlap goes: the call fails later, as there is no GPU."""
    return rc == 4


def test_linear_refuses_an_output_over_an_input(L):
    at = 1 << 24

    def call(x=1 << 30, xs=256, sx=None, M=4, K=256, w=1 << 32, sw=1 << 33, N=64, y=at, ys=64, t=0):
        return L.fl_int8_linear(ctypes.c_void_p(x), xs, ctypes.c_void_p(sx) if sx else None, M, K, ctypes.c_void_p(w), ctypes.c_void_p(sw),
                                N, ctypes.c_void_p(y), ys, t, ctypes.c_void_p(1 << 34), 1 << 40, None)
    for t, size in ((0, 2), (1, 4)):
        for M in (4, 1, 40):
            end = M * 64 * size                               # bytes of y, rows without gaps
            for d in (0, 16, -16, end - 16):                  # w, the scales, x: y's range meets theirs
                assert call(w=at + d, M=M, t=t) == 1 and call(sw=at + d, M=M, t=t) == 1 and call(x=at + d, M=M, t=t) == 1
                assert call(x=at + d, sx=1 << 35, M=M, t=t) == 1
            assert call(sx=at + end - 4, M=M, t=t) == 1 and call(sx=at - 4 * M + 4, M=M, t=t) == 1
            assert call(w=at - 64 * 256 + 16, M=M, t=t) == 1 and call(sw=at - 64 * 4 + 4, M=M, t=t) == 1
    # columns of one wide matrix: x in the first 256 of 320, y behind them or over their end
    for M in (1, 4, 40):
        assert call(x=at, xs=320, y=at + 2 * 255, ys=320, M=M) == 1 and call(x=at, xs=320, y=at - 2, ys=320, M=M) == 1
        if not torch.cuda.is_available():                     # (the addresses are no memory)
            assert _runs(call(x=at, xs=320, y=at + 2 * 256, ys=320, M=M)) and _runs(call(x=at + 2 * 64, xs=320, ys=320, M=M))
            assert _runs(call(x=at + 4 * 64 * M, M=M)) and _runs(call(w=at + 2 * 64 * M, M=M)) and _runs(call(w=at - 64 * 256, M=M))
            assert _runs(call(sw=at - 64 * 4, M=M)) and _runs(call(sx=at + 2 * 64 * M, M=M))
    assert call(x=at, xs=320, y=at + 4 * 200, ys=320, t=1) == 1   # strides of 640 and 1280 bytes that meet


def test_quantize_refuses_outputs_that_meet(L):
    at, far, M, K = 1 << 24, 1 << 30, 4, 64

    def call(x=at, xs=64, c=far, s=1 << 31):
        return L.fl_int8_quantize(ctypes.c_void_p(x), xs, M, K, ctypes.c_void_p(c), ctypes.c_void_p(s), None)
    for d in (0, 64, 511, -255):
        assert call(c=at + d) == 1
    assert call(s=at) == 1 and call(s=at + 508) == 1 and call(s=at - 12) == 1 and call(s=far) == 1 and call(s=far + 252) == 1
    if not torch.cuda.is_available():
        assert _runs(call()) and _runs(call(c=at + 512)) and _runs(call(c=at - 256)) and _runs(call(s=far + 256)) and _runs(call(s=far - 16))


# --------------------------------------------------------------- devices

class On:
    """A tensor that says it lies on a CUDA device."""
    is_cuda = True

    def __init__(self, t, index=0):
        self.t, self.index = t, index
        self.device = torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index

    def __getitem__(self, i):
        return On(self.t[i], self.index)


def _empty(shape, dtype=None, device=None):
    return On(torch.empty(shape, dtype=dtype))


def _zeros(*shape, dtype=torch.int32):
    return On(torch.zeros(shape, dtype=dtype))


@pytest.fixture
def gpu0(monkeypatch):
    """The binding as on a machine with GPUs, of which 0 is the current one; returns the
    library's calls, none of which runs."""
    calls = []

    def entry(name):
        if name.endswith("_workspace"):
            return lambda *a: 0
        return lambda *a: calls.append(name) or 0
    library = type("L", (), {"__getattr__": lambda self, name: entry(name)})()
    state = {"capturing": False}
    fake = types.SimpleNamespace(empty=_empty, empty_like=lambda t: On(torch.empty_like(t.t)),
                                 zeros=lambda n, dtype=None, device=None: On(torch.zeros(n, dtype=dtype)),
                                 _C=types.SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda i: 77),
                                 cuda=types.SimpleNamespace(is_current_stream_capturing=lambda: state["capturing"]),
                                 **{n: getattr(torch, n) for n in ("int8", "uint8", "int32", "float32", "float64", "bfloat16")})
    monkeypatch.setattr(fl, "_TORCH", fake)
    monkeypatch.setattr(fl, "lib", lambda: library)
    monkeypatch.setattr(fl, "_WS", {})
    monkeypatch.setattr(fl, "_OUTGROWN", [])
    return types.SimpleNamespace(calls=calls, state=state)


def _calls():
    """Every serving call with all of its tensors: (name, function, arguments)."""
    f32, bf16, u8, i8 = torch.float32, torch.bfloat16, torch.uint8, torch.int8
    ws = dict(ws=_zeros(4096, dtype=u8))
    pool = dict(refs=_zeros(6), table=_zeros(3, 4), kv_lens=_zeros(3))
    status = dict(status=_zeros(4))

    def copy(**kw):
        lists = [[kw.pop(f"{name}{i}") for i in range(2)] for name in ("k", "v", "a", "b")]
        return fl.fl_kv8_pages_copy(*lists, **kw)
    caches = {f"{name}{i}": _zeros(6, 1, 16, 64, dtype=u8) if name in "kv" else _zeros(6, 1, dtype=f32) for i in range(2) for name in "kvab"}
    return [
        ("quantize", fl.fl_int8_quantize, dict(x=_zeros(2, 32, dtype=bf16)), {}),
        ("linear", fl.fl_int8_linear, dict(x=_zeros(2, 32, dtype=bf16), w=_zeros(4, 32, dtype=i8), w_scale=_zeros(4, dtype=f32),
                                           y=_zeros(2, 4, dtype=bf16), **ws), {}),
        ("linear", fl.fl_int8_linear, dict(x=_zeros(2, 32, dtype=i8), x_scale=_zeros(2, dtype=f32), w=_zeros(4, 32, dtype=i8),
                                           w_scale=_zeros(4, dtype=f32)), {}),
        ("logits", fl.fl_logits_process, dict(
            logits=_zeros(2, 40, dtype=f32), history=_zeros(2, 8), history_lens=_zeros(2), prompt_lens=_zeros(2),
            repetition=_zeros(2, dtype=f32), frequency=_zeros(2, dtype=f32), presence=_zeros(2, dtype=f32), bias_offsets=_zeros(3),
            bias_ids=_zeros(5), bias=_zeros(5, dtype=f32), allowed=_zeros(2, 2), temperature=_zeros(2, dtype=f32),
            out=_zeros(2, 40, dtype=f32), **ws), {}),
        ("free", fl.fl_kv8_pages_free, dict(**pool, seqs=_zeros(2), keep=_zeros(2), **status), dict(block=16)),
        ("fork", fl.fl_kv8_pages_fork, dict(**pool, parents=_zeros(2), children=_zeros(2), **status), dict(block=16)),
        ("alloc", fl.fl_kv8_pages_alloc, dict(**pool, seqs=_zeros(2), new_tokens=_zeros(2), **ws), dict(block=16)),
        ("compact", fl.fl_kv8_pages_compact, dict(**pool, **status), dict(block=16)),
        ("copy", copy, dict(**caches, pairs=_zeros(2, 2), count=_zeros(1), **status), {}),
    ]


@pytest.mark.parametrize("which", range(9))
def test_tensors_of_another_device_are_refused(gpu0, which):
    name, call, tensors, rest = _calls()[which]
    call(**tensors, **rest)
    assert len(gpu0.calls) == 1 and name in gpu0.calls[0]
    for other, t in tensors.items():
        with pytest.raises(ValueError):
            call(**{**tensors, other: On(t.t, 1)}, **rest)
    with pytest.raises(ValueError):
        call(**{k: On(t.t, 1) for k, t in tensors.items()}, **rest)      # all on one that is not the current one
    assert len(gpu0.calls) == 1


# ---------------------------------------------------------- status blocks

@pytest.mark.parametrize("which", [4, 5, 7, 8])
def test_status_blocks_of_captured_calls_live_until_the_launch(gpu0, monkeypatch, which):
    """Without a status block a captured call makes one; it is not given back before
    the library has it."""
    made, alive = [], []
    name, call, tensors, rest = _calls()[which]
    zeros = fl._TORCH.zeros

    def noted(*a, **kw):
        t = zeros(*a, **kw)
        made.append(weakref.ref(t))
        return t
    fl._TORCH.zeros = noted
    library = type("L", (), {"__getattr__": lambda self, n: lambda *a: alive.append([r() is not None for r in made]) or 0})()
    monkeypatch.setattr(fl, "lib", lambda: library)
    gpu0.state["capturing"] = True
    call(**{**tensors, "status": None}, **rest)
    assert alive == [[True]]
