"""Host side of the serving operators (linear in 8-bit integers, logits' rules,
pages of the 8-bit cache): refusals before any launch, the binding's checks and
structures, and pins of their oracle.  No GPU."""
import ctypes
import random

import numpy as np
import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from int4_group_quantized_int4g_gb300 import _build
from oracle import serving_oracle as O

A = ctypes.c_void_p(0x10000)       # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)
HALF = ctypes.c_void_p(0x10002)
BYTE = ctypes.c_void_p(0x10001)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fl.lib()


def test_structures():
    assert ctypes.sizeof(fl.FlLogitsRules) == fl._LOGITS_RULES.size == 112
    assert ctypes.sizeof(fl.FlKv8Pool) == fl._KV8_POOL.size == 40
    assert ctypes.sizeof(fl.FlKv8Cache * 3) == fl._kv8_caches(3).size


def test_int8_quantize_refusals(L):
    def call(x=A, xs=64, M=2, K=64, c=A, s=A):
        return L.fl_int8_quantize(x, xs, M, K, c, s, None)
    assert call(x=None) == 1 and call(c=None) == 1 and call(s=None) == 1
    assert call(M=0) == 1 and call(K=0) == 1 and call(xs=63) == 1
    assert call(x=BYTE) == 1 and call(s=HALF) == 1


def test_int8_linear_refusals(L):
    size = ctypes.c_size_t(0)
    for M in (1, 16, 17, 300, 9000):
        assert L.fl_int8_linear_workspace(M, 1000, 272, ctypes.byref(size)) == 0 and size.value > M * 272 * 2
    assert L.fl_int8_linear_workspace(1, 1000, 264, ctypes.byref(size)) == 1       # K % 16
    assert L.fl_int8_linear_workspace(0, 1000, 256, ctypes.byref(size)) == 1
    assert L.fl_int8_linear_workspace(1, 0, 256, ctypes.byref(size)) == 1
    assert L.fl_int8_linear_workspace(1, 8, 256, None) == 1

    def call(x=A, xs=256, sx=None, M=2, K=256, w=A, sw=A, N=100, y=A, ys=100, t=0, ws=A, wb=BIG):
        return L.fl_int8_linear(x, xs, sx, M, K, w, sw, N, y, ys, t, ws, wb, None)
    for kw in (dict(x=None), dict(w=None), dict(sw=None), dict(y=None), dict(ws=None)):
        assert call(**kw) == 1
    assert call(K=250) == 1 and call(M=0) == 1 and call(N=0) == 1
    assert call(xs=255) == 1 and call(ys=99) == 1 and call(t=2) == 1
    assert call(w=ODD) == 1 and call(ws=ODD) == 1 and call(sw=HALF) == 1
    assert call(x=BYTE) == 1 and call(y=BYTE) == 1 and call(y=HALF, t=1) == 1
    assert call(sx=HALF) == 1
    for M in (2, 200):
        assert L.fl_int8_linear_workspace(M, 100, 256, ctypes.byref(size)) == 0
        assert call(M=M, wb=size.value - 1) == 2


def _walk(p, c):
    """The runs of units (tile, first, end) of pair c."""
    per, units = p["G"], p["units"]
    if p["whole"]:
        u = min(c, units // per) * per
        end = min(u + per, units)
    else:
        u, end = (c * units // p["P"], (c + 1) * units // p["P"]) if units else (0, 0)
    while u < end:
        t = u // per
        n = min(per - u % per, end - u)
        yield p["waves"] * p["P"] + t, u % per, u % per + n
        u += n
    for w in range(p["waves"]):
        yield w * p["P"] + c, 0, per


@pytest.mark.parametrize("sms", [152, 148, 20, 2])
def test_linear_plans_do_every_unit_once(L, sms):
    for M in (17, 24, 33, 64, 100, 128, 129, 301, 512, 700, 1000, 2048, 8190, 30000):
        for N, K in ((1, 16), (300, 4096), (4096, 4096), (11008, 4096), (4096, 11008), (16000, 512), (128003, 256)):
            p = fl.fl_int8_test_plan(M, N, K, sms)
            tiles = p["mtiles"] * p["ntiles"]
            assert 32 <= p["BN"] <= 256 and p["BN"] % 32 == 0 and (p["mtiles"] - 1) * p["BN"] < M <= p["mtiles"] * p["BN"]
            assert p["G"] == -(-K // 128) and p["ntiles"] == -(-N // 256) and 1 <= p["P"] <= sms // 2
            assert p["waves"] * p["P"] * p["G"] + p["units"] == tiles * p["G"]
            assert not p["units"] or p["whole"] or p["units"] >= p["P"]      # every run has a unit
            assert not p["whole"] or p["units"] <= p["P"] * p["G"]
            done = {}
            for c in range(p["P"]):
                for t, a, b in _walk(p, c):
                    assert 0 <= t < tiles and a < b
                    done.setdefault(t, []).append((a, b))
            assert len(done) == tiles
            for runs in done.values():
                runs.sort()
                assert runs[0][0] == 0 and runs[-1][1] == p["G"] and all(x[1] == y[0] for x, y in zip(runs, runs[1:]))


def _rules(**kw):
    d = dict(history=0x10000, history_lens=0x10000, prompt_lens=0x10000, repetition=0x10000, frequency=0x10000, presence=0x10000,
             bias_offsets=0x10000, bias_ids=0x10000, bias=0x10000, allowed=0x10000, temperature=0x10000, history_stride=50,
             allowed_stride=4, history_max=50, bias_count=7)
    d.update(kw)
    return ctypes.byref(fl.FlLogitsRules(**d))


def test_logits_refusals(L):
    size = ctypes.c_size_t(0)
    assert L.fl_logits_process_workspace(3, 100, ctypes.byref(size)) == 0 and size.value > 0
    assert L.fl_logits_process_workspace(0, 100, ctypes.byref(size)) == 1
    assert L.fl_logits_process_workspace(3, 0, ctypes.byref(size)) == 1
    assert L.fl_logits_process_workspace(3, 1 << 30, ctypes.byref(size)) == 1

    def call(x=A, xs=100, t=1, B=3, V=100, r=None, out=A, os_=100, tok=A, lse=A, lp=A, ws=A, wb=BIG):
        return L.fl_logits_process(x, xs, t, B, V, r or _rules(), out, os_, tok, lse, lp, ws, wb, None)
    assert L.fl_logits_process(A, 100, 1, 3, 100, None, A, 100, A, A, A, A, BIG, None) == 1
    assert call(x=None) == 1 and call(tok=None) == 1 and call(ws=None) == 1
    assert call(B=0) == 1 and call(V=0) == 1 and call(t=2) == 1
    assert call(xs=99) == 1 and call(os_=99) == 1
    assert call(x=HALF) == 1 and call(out=HALF) == 1 and call(tok=BYTE) == 1 and call(ws=ODD) == 1
    assert call(t=0) == 1 and call(os_=101) == 1                     # in place: the same type and stride
    assert call(out=ctypes.c_void_p(0x10000 + 4), os_=100) == 1      # a row over itself, shifted
    assert call(xs=300, os_=300, out=ctypes.c_void_p(0x10000 + 4 * 250)) == 1     # over the next row
    assert call(xs=300, os_=200, out=ctypes.c_void_p(0x10000 + 4 * 150)) == 1
    other = ctypes.c_void_p(0x90000)
    for bad in (dict(history_lens=None), dict(history=None), dict(history_stride=49), dict(history_max=-1), dict(history_max=1 << 30),
                dict(history=None, history_lens=None), dict(bias=None), dict(bias_ids=None), dict(bias_offsets=None),
                dict(bias_count=-1), dict(allowed_stride=3), dict(temperature=0x10002), dict(history=0x10001)):
        assert call(out=other, r=_rules(**bad)) == 1, bad
    assert call(out=other, wb=64) == 2


def _pool(**kw):
    d = dict(refs=0x10000, table=0x10000, kv_lens=0x10000, num_blocks=8, slots=4, max_blocks=3, block=16)
    d.update(kw)
    return ctypes.byref(fl.FlKv8Pool(**d))


def test_pages_refusals(L):
    size = ctypes.c_size_t(0)
    assert L.fl_kv8_pages_workspace(_pool(), ctypes.byref(size)) == 0 and size.value > 0
    assert L.fl_kv8_pages_workspace(_pool(), None) == 1
    calls = {
        "free": lambda p=None, a=A, b=A, n=2, st=A: L.fl_kv8_pages_free(p or _pool(), a, b, n, st, None),
        "fork": lambda p=None, a=A, b=A, n=2, st=A: L.fl_kv8_pages_fork(p or _pool(), a, b, n, st, None),
        "alloc": lambda p=None, a=A, b=A, n=2, st=A: L.fl_kv8_pages_alloc(p or _pool(), a, b, n, A, A, A, st, BIG, None),
    }
    for name, call in calls.items():
        for bad in (dict(refs=None), dict(table=None), dict(kv_lens=None), dict(num_blocks=0), dict(slots=0), dict(max_blocks=0),
                    dict(refs=0x10002)):
            assert call(p=_pool(**bad)) == 1, (name, bad)
        for bad in (dict(block=24), dict(block=0), dict(slots=1 << 20, max_blocks=1 << 20)):
            assert call(p=_pool(**bad)) == 3, (name, bad)
        assert call(a=None) == 1 and call(a=HALF) == 1 and call(n=-1) == 1 and call(st=None) == 1 and call(st=ODD) == 1, name
        assert call(b=HALF) == 1, name
    assert L.fl_kv8_pages_fork(_pool(), A, None, 2, A, None) == 1
    assert L.fl_kv8_pages_alloc(_pool(), A, A, 2, A, A, A, A, size.value - 1, None) == 2
    for i in range(3):
        outs = [A, A, A]
        outs[i] = None
        assert L.fl_kv8_pages_alloc(_pool(), A, A, 2, *outs, A, BIG, None) == 1

    def compact(p=None, t=A, r=A, m=A, pr=A, c=A, st=A):
        return L.fl_kv8_pages_compact(p or _pool(), t, r, m, pr, c, st, None)
    assert all(compact(**{k: None}) == 1 for k in ("t", "r", "m", "pr", "c", "st"))
    assert compact(p=_pool(block=17)) == 3

    def cache(**kw):
        d = dict(k=0x10000, v=0x10000, k_scale=0x10000, v_scale=0x10000, num_blocks=8, block=16, kv_heads=2, head_dim=64, format=0)
        d.update(kw)
        return fl.FlKv8Cache(**d)

    def copy(c=None, layers=1, pr=A, n=A, most=3, st=A):
        arr = (fl.FlKv8Cache * 2)(*(c or [cache(), cache()]))
        return L.fl_kv8_pages_copy(arr, layers, pr, n, most, st, None)
    assert copy(layers=0) == 1 and copy(pr=None) == 1 and copy(n=None) == 1 and copy(most=-1) == 1 and copy(st=None) == 1
    assert copy([cache(k=None), cache()]) == 1 and copy([cache(v=0x10008), cache()]) == 1 and copy([cache(k_scale=None), cache()]) == 1
    assert copy([cache(), cache(num_blocks=9)], 2) == 1 and copy([cache(), cache(head_dim=128)], 2) == 1
    assert copy([cache(block=20), cache()]) == 3 and copy([cache(head_dim=96), cache()]) == 3
    assert copy([cache(num_blocks=1 << 28), cache()]) == 3


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros((2, 32), dtype=torch.bfloat16)
    w, t = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError):
        fl.fl_int8_quantize(x[0])
    with pytest.raises(ValueError):
        fl.fl_int8_linear(x, w[:, :16], t)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        fl.fl_int8_linear(x, w, t)
    with pytest.raises(ValueError):
        fl.fl_logits_process(torch.zeros(5))
    one = [torch.zeros((1, 1, 16, 64), dtype=torch.uint8)]
    with pytest.raises(ValueError):
        fl.fl_kv8_pages_copy(one, [], one, one, x, x)


# ------------------------------------------------------------ the oracle

def test_oracle_quantize8_by_fractions():
    from fractions import Fraction
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((20, 40)).astype(np.float32)).to(torch.bfloat16).double().numpy()
    x[3, 5] = 127 * 0.5
    x[3, 6] = 0.25                     # a quotient of 1/2 by a scale of 1/2: to even
    q, s = O.quantize8(x)
    for m in range(20):
        assert np.float32(s[m]) == np.float32(np.abs(x[m]).max()) / np.float32(127)
        for k in range(40):
            exact = Fraction(x[m, k]) / Fraction(s[m])
            assert abs(exact - int(q[m, k])) <= Fraction(1, 2)
            if abs(exact - int(q[m, k])) == Fraction(1, 2):
                assert q[m, k] % 2 == 0
    assert q[3, 6] == 0


def test_oracle_logits_hand_case():
    x = np.array([[1.0, -2.0, 3.0, 0.0, 3.0]])
    got, token, lse, logprob = O.logits(
        x, history=np.array([[2, 1, 2, 2, 7]]), history_lens=[5], prompt_lens=[1], repetition=[2.0], frequency=[0.25], presence=[0.5],
        bias_offsets=[0, 3], bias_ids=[3, 3, -1], bias=[1.0, 2.0, 9.0], allowed=np.array([[0b01111]]), temperature=[0.5])
    # 1: -2 * 2 - 0.25 - 0.5; 2: 3 / 2 - 2 * 0.25 - 0.5; 3: + 3; 4 is masked; all times 2
    want = np.array([2.0, -9.5, 1.0, 6.0, -np.inf])
    assert np.allclose(got[0], want) and token[0] == 3
    assert np.isclose(lse[0], np.log(np.exp(want).sum())) and np.isclose(logprob[0], 6.0 - lse[0])
    got, token, lse, logprob = O.logits(np.zeros((1, 40)), allowed=np.zeros((1, 2), dtype=np.int32))
    assert token[0] == -1 and lse[0] == logprob[0] == -np.inf


def test_oracle_pool_keeps_its_books():
    """After any run of calls a page's holders are the sequences whose tables name it."""
    rng = random.Random(1)
    p = O.Pool(30, 9, 5, 16)
    for _ in range(400):
        order = rng.sample(range(9), rng.randint(1, 9))
        what = rng.randrange(5)
        if what < 2:
            _, pairs = p.alloc(order, [min(rng.choice([0, 1, 3, 20]), 80 - p.lens[s]) for s in order])
            assert all(p.refs[t] == 1 for _, t in pairs)
        elif what == 2:
            p.free(order, [rng.randint(0, 80) for _ in order])
        elif what == 3:
            full = [s for s in range(9) if p.lens[s]]
            if full:
                p.fork([rng.choice(full) for _ in order], order)
        else:
            live = sum(r > 0 for r in p.refs)
            p.compact()
            assert all(r > 0 for r in p.refs[:live]) and not any(p.refs[live:])
        held = [0] * 30
        for s, n in enumerate(p.lens):
            for page in p.table[s][:p.pages(n)]:
                held[page] += 1
        assert held == p.refs
        for s, n in enumerate(p.lens):    # a page that is written next is held by nobody else, or has been copied
            assert len(set(p.table[s][:p.pages(n)])) == p.pages(n)
