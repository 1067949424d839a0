"""GPU parity of the linear in 8-bit integers, the logits' rules with the choice
of a token, and the pages of the 8-bit cache, against the float64 oracle.

Whole numbers have to be equal.  Tolerances count roundings: half a step of bf16
is 2^-8 of the value (its spacing relative to the value's lower end), of fp32
2^-24."""
import numpy as np
import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from oracle import serving_oracle as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int4_group_quantized_int4g_gb300 import _build
    _build.build()
    fl.lib()


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def _f32(a):
    return torch.tensor(np.asarray(a, dtype=np.float32), device=DEV)


# ---------------------------------------------------------------- quantize

def _codes_check(x):
    codes, scale = fl.fl_int8_quantize(x)
    q, s = O.quantize8(_np(x))
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.array_equal(_np(scale), s, equal_nan=True)


@pytest.mark.parametrize("K", [1, 7, 8, 16, 100, 256, 1000, 4096, 5001, 8200, 33000, 70001])
@pytest.mark.parametrize("M", [1, 5, 400])
def test_quantize_widths(K, M):
    if M * K > 3000000:
        M = 40
    rng = np.random.default_rng(K + M)
    _codes_check(_bf16(rng.standard_normal((M, K)) * 10.0 ** rng.integers(-6, 6, (M, 1))).to(DEV))


def test_quantize_borders():
    """Rows whose quotients lie on borders, or as near as bf16 and fp32 let them."""
    rows = []
    for top in (127.0, 254.0, 1.984375, 2.0 ** -130, 2.0 ** -133, 3.0e38, 2.0 ** -60 * 127, 2.0 ** -61 * 127):
        step = top / 127
        row = (np.arange(256) - 128 + 0.5) * step
        row = np.clip(row, -top, top)
        row[0] = top
        rows.append(row)
    rng = np.random.default_rng(5)
    for e in range(-130, 128, 3):
        row = rng.integers(-127, 128, 256) * 2.0 ** (e - 8)
        row[0] = 2.0 ** e * 0.99
        rows.append(row)
    _codes_check(_bf16(np.array(rows)).to(DEV))


@pytest.mark.parametrize("e", [-133, -126, -60, 0, 99, 100, 127])
def test_quantize_every_value_of_a_binade_over_every_top(e):
    """Rows of all bf16 values that a largest value of binade e can meet in its own and the next binades."""
    tops = (128 + np.arange(0, 128, 3)) * 2.0 ** max(e - 7, -140)
    values = np.concatenate([(128 + np.arange(128)) * 2.0 ** max(e - 7 - i, -140 - i) for i in range(7)])
    rows = np.minimum(values[None], tops[:, None]) * np.where(np.arange(len(values)) % 2, -1.0, 1.0)
    rows[:, 0] = tops
    _codes_check(_bf16(rows).to(DEV))


def test_quantize_zeros_and_infinities():
    x = torch.ones((5, 300), dtype=torch.bfloat16, device=DEV)
    x[0] = 0
    x[1, 7] = float("inf")
    x[2, 299] = float("nan")
    x[3, 0] = float("-inf")
    x[4] = -0.0
    _codes_check(x)


def test_quantize_rows_of_a_wider_matrix():
    rng = np.random.default_rng(11)
    wide = _bf16(rng.standard_normal((9, 700))).to(DEV)
    for lo, hi in ((8, 520), (3, 600), (0, 512)):
        _codes_check(wide[:, lo:hi])


# ------------------------------------------------------------------ linear

def _linear_case(M, N, K, seed, same_sign=False):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp(0.5 * rng.standard_normal((1, K)))
    w = rng.integers(-128, 128, (N, K))
    if same_sign:
        x, w = np.abs(x), np.abs(np.maximum(w, -127))
    t = np.exp(0.3 * rng.standard_normal(N)) * 1e-3
    return _bf16(x).to(DEV), torch.from_numpy(w.astype(np.int8)).to(DEV), _f32(t)


def _linear_check(y, q, s, w, t, K):
    dot, scale = O.linear8(q, s, w.cpu().numpy(), _np(t))
    ref = dot * scale
    # sums of whole numbers are exact below 2^24; above, each of the K / 16 steps
    # of a sum (and of joining the parts) rounds by at most a step, 2^-23 of it
    mag = np.abs(q.astype(np.float64)) @ np.abs(w.cpu().numpy().astype(np.float64)).T
    tol = np.where(mag < 2 ** 24, 0.0, mag * (K / 16 + 20) * 2.0 ** -23) * np.abs(scale)
    tol += np.abs(ref) * (2.0 ** -8 if y.dtype == torch.bfloat16 else 0) + np.abs(ref) * 3 * 2.0 ** -24 + 1e-44
    assert np.all(np.abs(_np(y) - ref) <= tol), np.max(np.abs(_np(y) - ref) / tol)


SIZES = [(1, 1, 16), (1, 100, 256), (3, 256, 128), (1, 4096, 1024), (7, 1000, 4096), (8, 300, 144), (9, 257, 1040), (16, 513, 272),
         (17, 128, 2064), (20, 600, 384), (48, 1500, 1536), (65, 700, 2176), (96, 300, 640), (24, 5003, 512), (31, 255, 1024), (32, 700, 4096), (32, 40000, 256), (1, 300, 28672), (2, 40007, 896),
         (33, 127, 128), (40, 1000, 1040), (64, 4096, 512), (100, 129, 16), (128, 2500, 1008), (150, 300, 4096), (257, 777, 400),
         (301, 1100, 2048), (512, 200, 6144), (700, 2049, 272), (1111, 130, 1024), (2050, 384, 528),
         (2048, 4864, 144), (2304, 4870, 272), (3000, 5000, 256), (301, 11008, 272), (700, 4096, 400), (64, 11008, 144),
         (512, 11008, 272)]   # whole waves of tiles: without a rest, and with one


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_sizes(M, N, K):
    x, w, t = _linear_case(M, N, K, M * 7 + N * 3 + K)
    q, s = O.quantize8(_np(x))
    for dtype in (torch.bfloat16, torch.float32):
        y = fl.fl_int8_linear(x, w, t, out_dtype=dtype)
        assert y.shape == (M, N) and y.dtype == dtype
        _linear_check(y, q, s, w, t, K)
    codes, scale = fl.fl_int8_quantize(x)
    assert torch.equal(fl.fl_int8_linear(codes, w, t, x_scale=scale, out_dtype=torch.float32), y)


@pytest.mark.parametrize("M", [1, 30, 200])
def test_linear_large_sums(M):
    """Sums past 2^24: all products of one sign."""
    x, w, t = _linear_case(M, 300, 8192, M, same_sign=True)
    q, s = O.quantize8(_np(x))
    _linear_check(fl.fl_int8_linear(x, w, t, out_dtype=torch.float32), q, s, w, t, 8192)


@pytest.mark.parametrize("M", [2, 32, 45, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_strides_and_guards(M, dtype):
    """x and y as columns of wider matrices, aligned and not; nothing beside y is touched."""
    N, K = 333, 272
    x, w, t = _linear_case(M, N, K, M)
    want = fl.fl_int8_linear(x, w, t, out_dtype=dtype)
    codes, scale = fl.fl_int8_quantize(x)
    for lead, width in ((0, 512), (8, 600), (5, 601), (3, 1000)):
        wide = torch.full((M, width), 7.0, dtype=torch.bfloat16, device=DEV)
        wide[:, lead:lead + K] = x
        out = torch.full((M + 2, width), -3.0, dtype=dtype, device=DEV)
        y = out[1:M + 1, lead:lead + N]
        assert fl.fl_int8_linear(wide[:, lead:lead + K], w, t, y=y) is y
        assert torch.equal(y, want)
        y.fill_(-3.0)
        assert bool((out == -3.0).all())
        wide8 = torch.zeros((M, width), dtype=torch.int8, device=DEV)
        wide8[:, lead:lead + K] = codes
        assert torch.equal(fl.fl_int8_linear(wide8[:, lead:lead + K], w, t, x_scale=scale, out_dtype=dtype), want)


@pytest.mark.parametrize("M", [3, 70])
def test_linear_rows_without_a_scale(M):
    """A token with an infinity is NaN throughout, one of zeros is 0; the others are as they were."""
    x, w, t = _linear_case(M, 500, 256, 3)
    want = fl.fl_int8_linear(x, w, t)
    x[0, 5], x[1] = float("inf"), 0
    y = fl.fl_int8_linear(x, w, t)
    assert bool(y[0].isnan().all()) and not y[1].any() and torch.equal(y[2:], want[2:])


def test_linear_repeats_streams_and_graphs():
    """The same bits each time, on another stream, and replayed with new inputs."""
    for M, N, K in ((1, 4096, 4096), (20, 3000, 2048), (90, 1500, 1024), (300, 2000, 1040)):
        x, w, t = _linear_case(M, N, K, M)
        x2 = _linear_case(M, N, K, M + 1)[0]
        want, want2 = fl.fl_int8_linear(x, w, t), fl.fl_int8_linear(x2, w, t)
        for _ in range(5):
            assert torch.equal(fl.fl_int8_linear(x, w, t), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = fl.fl_int8_linear(x, w, t)
        side.synchronize()
        assert torch.equal(y, want)
        ws = torch.zeros(fl.fl_int8_linear_workspace(M, N, K), dtype=torch.uint8, device=DEV)
        xin, y = x.clone(), torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fl.fl_int8_linear(xin, w, t, y=y, ws=ws)
        for src, ref in ((x2, want2), (x, want)):
            xin.copy_(src)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, ref)
        assert fl.fl_int4g_status(ws) == 0


def test_linear_workspace_is_enough():
    for M, N, K in ((1, 300, 4096), (32, 5000, 512), (200, 700, 1040), (500, 3000, 256)):
        x, w, t = _linear_case(M, N, K, M)
        n = fl.fl_int8_linear_workspace(M, N, K)
        guard = torch.full((n + 4096,), 0, dtype=torch.uint8, device=DEV)
        guard[n:] = 0xA5
        fl.fl_int8_linear(x, w, t, ws=guard[:n])
        assert bool((guard[n:] == 0xA5).all())


# ------------------------------------------------------------------ logits

def _logits_case(B, V, seed, dtype, history=0, biases=0, grammar=False):
    rng = np.random.default_rng(seed)
    x = (3 * rng.standard_normal((B, V))).astype(np.float32)
    x = torch.from_numpy(x).to(DEV).to(dtype)
    kw = {}
    if history:
        few = rng.integers(0, V, (B, 20))
        h = np.where(rng.random((B, history)) < 0.5, np.take_along_axis(few, rng.integers(0, 20, (B, history)), 1),
                     rng.integers(0, V, (B, history)))
        kw["history"] = h.astype(np.int32)
        kw["history_lens"] = rng.integers(0, history + 1, B).astype(np.int32)
        kw["history_lens"][0] = history
        kw["prompt_lens"] = (kw["history_lens"] * rng.random(B)).astype(np.int32)
        kw["repetition"] = (1 + 0.3 * np.abs(rng.standard_normal(B))).astype(np.float32)
        kw["frequency"] = (0.2 * rng.standard_normal(B)).astype(np.float32)
        kw["presence"] = (0.4 * rng.standard_normal(B)).astype(np.float32)
    if biases:
        kw["bias_offsets"] = (np.arange(B + 1) * biases).astype(np.int32)
        kw["bias_ids"] = rng.integers(0, V, B * biases).astype(np.int32)
        kw["bias"] = (5 * rng.standard_normal(B * biases)).astype(np.float32)
    if grammar:
        kw["allowed"] = (rng.integers(-2 ** 31, 2 ** 31, (B, -(-V // 32))) & rng.integers(-2 ** 31, 2 ** 31, (B, -(-V // 32)))
                         ).astype(np.int32)
    kw["temperature"] = (0.4 + np.abs(rng.standard_normal(B))).astype(np.float32)
    return x, kw


def _logits_check(x, kw, got=None):
    if got is None:
        got = fl.fl_logits_process(x, **{k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in kw.items()})
    with np.errstate(all="ignore"):
        want, token, lse, logprob = O.logits(x.float().cpu().numpy(), **kw, real=np.float32)
    if "logits" in got:
        assert np.array_equal(got["logits"].cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(got["token"].cpu().numpy(), token)
    # exp is good to 2^-22 and |x - max| 2^-23, their sum to 2^-20 with its additions; the logarithm turns
    # that into an absolute error, and is itself good to 2^-22 of its size
    ok = np.isfinite(lse)
    for name, ref in (("lse", lse), ("logprob", logprob)):
        v = _np(got[name])
        assert np.array_equal(v[~ok], ref[~ok], equal_nan=True), name
        assert np.all(np.abs(v[ok] - ref[ok]) <= 2.0 ** -18 + 2.0 ** -22 * (np.abs(ref[ok]) + np.abs(lse[ok]))), name


@pytest.mark.parametrize("V", [1, 2, 7, 31, 33, 100, 1023, 1024, 1025, 1031, 5000, 32000, 50257])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [1, 3])
def test_logits_sizes(V, dtype, B):
    x, kw = _logits_case(B, V, V + B, dtype)
    _logits_check(x, kw)
    _logits_check(x, {})
    x, kw = _logits_case(B, V, V + B, dtype, history=37, biases=5, grammar=True)
    _logits_check(x, kw)


@pytest.mark.parametrize("history,biases,grammar", [(1, 0, False), (0, 1, False), (0, 0, True), (3, 700, False), (5000, 0, True),
                                                    (70000, 30, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logits_rules(history, biases, grammar, dtype):
    _logits_check(*_logits_case(3, 20003, history + biases, dtype, history, biases, grammar))


@pytest.mark.parametrize("B,V", [(64, 32001), (300, 16390), (1300, 1000), (40, 130000)])
def test_logits_many_rows(B, V):
    """Long runs, one run a row, and several rows an SM."""
    _logits_check(*_logits_case(B, V, B, torch.float32, history=20, biases=3, grammar=True))
    x, kw = _logits_case(B, V, B + 1, torch.bfloat16, history=11)
    _logits_check(x, kw)


def test_logits_more_rows_than_tickets():
    """Rows in several launches: a long batch, one run a row and several."""
    for B, V in ((66000, 33), (65540, 1100)):
        x, kw = _logits_case(B, V, 1, torch.bfloat16, history=1)
        dev = {k: torch.from_numpy(v).to(DEV) for k, v in kw.items()}
        got = fl.fl_logits_process(x, **dev)
        some = np.concatenate([np.arange(0, B, 997), np.arange(65530, B)])
        _logits_check(x[torch.from_numpy(some).to(DEV)], {k: v[some] for k, v in kw.items()},
                      {k: v[torch.from_numpy(some).to(DEV)] for k, v in got.items()})


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logits_many_rows_of_several_runs(dtype):
    """As many CTAs as take a kernel of their own to join the runs: rows without a token, with a NaN, with the
    largest in several runs; the same bits replayed; then few rows with the same workspace."""
    B, V = 1000, 20003
    x, kw = _logits_case(B, V, 4, dtype, history=30, biases=3, grammar=True)
    x[3, 12345], x[4, 19999], x[5] = float("nan"), float("inf"), -float("inf")
    x[6, 50:20000:997] = 80.0
    kw["allowed"][6], kw["allowed"][7] = -1, 0
    kw["bias"][18:21] = 0
    dev = {k: torch.from_numpy(v).to(DEV) for k, v in kw.items()}
    ws = torch.zeros(fl.fl_logits_process_workspace(B, V), dtype=torch.uint8, device=DEV)
    got = fl.fl_logits_process(x, **dev, ws=ws)
    some = np.concatenate([np.arange(20), np.arange(20, B, 37), [B - 1]])
    at = torch.from_numpy(some).to(DEV)
    pick = {k: v[some] for k, v in kw.items() if not k.startswith("bias")}
    pick["bias_offsets"] = (3 * np.arange(len(some) + 1)).astype(np.int32)
    pick["bias_ids"], pick["bias"] = kw["bias_ids"].reshape(B, 3)[some].ravel(), kw["bias"].reshape(B, 3)[some].ravel()
    _logits_check(x[at], pick, {k: v[at] for k, v in got.items()})
    assert got["token"][5] == -1 and got["token"][7] == -1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = fl.fl_logits_process(x, **dev, ws=ws)
    for _ in range(3):
        for v in again.values():
            v.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for k, v in got.items():
        assert torch.equal(again[k].view(torch.int32), v.view(torch.int32)), k
    few, kf = _logits_case(3, V, 5, dtype, history=30)
    _logits_check(few, kf, fl.fl_logits_process(few, **{k: torch.from_numpy(v).to(DEV) for k, v in kf.items()}, ws=ws))
    assert fl.fl_int4g_status(ws) == 0


@pytest.mark.parametrize("V", [4097, 5000, 8191, 8192, 8193])
def test_logits_rows_of_one_long_run(V):
    _logits_check(*_logits_case(700, V, V, torch.float32, history=60, biases=2, grammar=True))
    _logits_check(*_logits_case(650, V, V + 1, torch.bfloat16, history=90))


def _logits_some(x, kw, biases, some, got):
    """The rows `some` of a call against the formula's; lists of biases of one length."""
    at = torch.from_numpy(some).to(DEV)
    pick = {k: v[some] for k, v in kw.items() if not k.startswith("bias")}
    if biases:
        pick["bias_offsets"] = (biases * np.arange(len(some) + 1)).astype(np.int32)
        pick["bias_ids"], pick["bias"] = (kw[k].reshape(-1, biases)[some].ravel() for k in ("bias_ids", "bias"))
    _logits_check(x[at], pick, {k: v[at] for k, v in got.items()})


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("history", [1023, 1999, 2048, 2501, 5003, 20000, 23040, 23041, 32768])
def test_logits_many_rows_with_histories(history, dtype):
    """Histories that are sorted by run first, in one launch or several, and those beside their limits: rows on and off
    16 bytes, padding, tokens outside the vocabulary, one token throughout, all of prompt or answer, none."""
    B, V = 1000, 20003
    x, kw = _logits_case(B, V, history, dtype, history=history, biases=2)
    h, lens, prompt = kw["history"], kw["history_lens"], kw["prompt_lens"]
    lens[1], prompt[1] = history, history
    lens[2], prompt[2] = history, 0
    h[2] = 17
    h[3, ::3], h[4, 1::2] = -1, V
    lens[3], lens[4] = history, history
    h[5] = np.arange(history) % 9           # the tokens before a row's first 16 bytes among them
    lens[5], lens[6], lens[7], prompt[8] = history, 0, -3, 2 * history
    h[9, 0], h[9, -1], lens[9] = V - 1, 2 ** 31 - 1, history
    h[10], lens[10] = np.where(np.arange(history) % 2, 4095 + np.arange(history) % 9, -2 ** 31), history + 5
    dev = {k: torch.from_numpy(v).to(DEV) for k, v in kw.items()}
    some = np.concatenate([np.arange(16), np.arange(16, B, 83), [418, 419, 420, 999]])
    got = fl.fl_logits_process(x, **dev)
    _logits_some(x, kw, 2, some, got)
    wide = torch.zeros((B, V + 14), dtype=dtype, device=DEV)[:, 3:3 + V]
    wide.copy_(x)
    other = fl.fl_logits_process(wide, **dev)
    for k, v in got.items():
        if k in ("logits", "token"):
            assert torch.equal(other[k], v), k
    _logits_some(wide, kw, 2, some[:16], other)


def test_logits_made_just_before_with_sorted_histories():
    """The logits by the kernel before, on another stream too, again and again, in place."""
    B, V, K = 700, 32000, 64
    w = torch.randint(-127, 128, (V, K), device=DEV, dtype=torch.int8)
    t = torch.full((V,), 1e-2, device=DEV)
    _, kw = _logits_case(B, V, 8, torch.float32, history=2400)
    dev = {k: torch.from_numpy(v).to(DEV) for k, v in kw.items()}
    xs = [torch.randn((B, K), device=DEV).to(torch.bfloat16) for _ in range(4)]
    want = []
    for x in xs:
        y = fl.fl_int8_linear(x, w, t, out_dtype=torch.float32)
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in fl.fl_logits_process(y, **dev).items()})
        torch.cuda.synchronize()
    y = torch.empty((B, V), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            for i in range(12):
                fl.fl_int8_linear(xs[i % 4], w, t, y=y)
                got = fl.fl_logits_process(y, **dev, out=y if i % 2 else None)
                for k, v in got.items():
                    assert torch.equal(v, want[i % 4][k]), (i, k)
        stream.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V", [(9, 2), (12, 33), (40, 5000), (30, 20003), (5, 128003), (900, 24001)])
def test_logits_logprob_of_nearly_certain_tokens(B, V, dtype):
    """One token far above the others: its log-probability is -log(1 + rest), good relative to itself."""
    rng = np.random.default_rng(V)
    x = torch.from_numpy((-14 - 8 * rng.random((B, V))).astype(np.float32)).to(DEV).to(dtype)
    spots = np.concatenate([[0, V - 1, V // 2], rng.integers(0, V, B)])[:B]
    at = torch.from_numpy(spots).to(DEV)
    x[torch.arange(B, device=DEV), at] = 1.0
    x[B - 1, V - 1 - spots[B - 1]] = 1.0            # (one row with two of them, mostly)
    got = fl.fl_logits_process(x)
    y = _np(x.float())
    rest = np.exp(y - 1).sum(1) - 1
    rest = np.where(rest > 0.5, rest, np.exp(np.where(y < 1, y, -np.inf) - 1).sum(1))
    # a term exp(d), |d| <= 24: three roundings of d, 2^-24 each, and exp's own 2^-22 make 2^-17.5; additions and
    # log1p fit into the rest of 2^-17
    assert np.all(np.abs(_np(got["logprob"]) + np.log1p(rest)) <= 2.0 ** -17 * np.log1p(rest))
    assert np.all(np.abs(_np(got["lse"]) - 1 - np.log1p(rest)) <= 2.0 ** -23 + 2.0 ** -17 * np.log1p(rest))
    assert np.array_equal(got["token"].cpu().numpy(), y.argmax(1))


def test_captured_calls_without_a_workspace():
    """Scratch is the graph's own and not cleared: the second replay finds what the first has left."""
    x, kw = _logits_case(700, 32000, 3, torch.float32, history=2400)
    dev = {k: torch.from_numpy(v).to(DEV) for k, v in kw.items()}
    a, w, t = _linear_case(90, 1500, 1024, 2)
    b = a[:1]
    want = fl.fl_logits_process(x, **dev), fl.fl_int8_linear(a, w, t), fl.fl_int8_linear(b, w, t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one, two, three = fl.fl_logits_process(x, **dev), fl.fl_int8_linear(a, w, t), fl.fl_int8_linear(b, w, t)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want[0].items():
            assert torch.equal(one[k], v), k
        assert torch.equal(two, want[1]) and torch.equal(three, want[2])
        for v in (*one.values(), two, three):
            v.zero_()


def test_logits_each_rule_alone():
    x, kw = _logits_case(4, 3001, 9, torch.float32, history=200, biases=9, grammar=True)
    base = {k: kw[k] for k in ("history", "history_lens")}
    for name in ("prompt_lens", "repetition", "frequency", "presence"):
        _logits_check(x, {**base, name: kw[name]})
    _logits_check(x, base)
    _logits_check(x, {k: kw[k] for k in ("bias_offsets", "bias_ids", "bias")})
    _logits_check(x, {"allowed": kw["allowed"]})
    _logits_check(x, {"temperature": np.array([0.0, -1.0, np.nan, 1e30], dtype=np.float32)})


def test_logits_biases_of_one_token_in_list_order():
    V = 9000
    x = torch.zeros((2, V), dtype=torch.float32, device=DEV)
    ids = np.array([5, 5, 8191, 5, 8999, 8191, -1, V, 7, 7], dtype=np.int32)
    b = np.array([1.0, 2.0 ** 24, 0.25, 1.0, 3.0, -0.25, 9.0, 9.0, 1e30, -1e30], dtype=np.float32)
    kw = {"bias_offsets": np.array([0, 8, 10], dtype=np.int32), "bias_ids": ids, "bias": b}
    _logits_check(x, kw)
    kw["bias_offsets"] = np.array([-5, 3, 99], dtype=np.int32)     # cut to the list
    _logits_check(x, kw)
    kw["bias_offsets"] = np.array([8, 3, 4], dtype=np.int32)       # falling: none
    _logits_check(x, kw)


def test_logits_histories_with_padding_and_odd_lengths():
    x, kw = _logits_case(6, 2000, 4, torch.float32, history=41)
    kw["history"][1, 5:9] = -1
    kw["history"][2, :] = 2000
    kw["history"][3, :] = 1999
    kw["history_lens"] = np.array([41, 41, 41, 41, 99999, -3], dtype=np.int32)
    kw["prompt_lens"] = np.array([0, 41, 3, 20, 99999, -1], dtype=np.int32)
    _logits_check(x, kw)


def test_logits_masked_rows_and_extreme_values():
    V = 5003
    x, kw = _logits_case(9, V, 5, torch.float32)
    words = np.full((9, -(-V // 32)), -1, dtype=np.int32)
    words[0] = 0                                 # nothing is left
    words[1] = 0
    words[1, 156] = 1 << 10                      # the token 5002, the last
    x[1, 5002] = -1e38
    x[2] = float("-inf")
    x[3, 17] = float("inf")
    x[4, 4000] = float("nan")
    x[5] = -3.4028234663852886e38                # the type's lowest everywhere: still tokens
    x[6, :] = 2.5                                # ties: the first
    x[7, 100] = x[7, 4999] = 50.0
    words[7, 3] = ~(1 << 4)                      # ... of those that are left
    x[8, 3], x[8, 4] = float("nan"), float("inf")
    words[8, 0] = ~0b11000                       # masked NaN and infinity are gone
    kw["allowed"] = words
    kw["temperature"] = np.ones(9, dtype=np.float32)
    _logits_check(x, kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logits_strides_in_place_and_without_an_output(dtype):
    B, V = 5, 3333
    x, kw = _logits_case(B, V, 8, dtype, history=50, biases=4, grammar=True)
    dev = {k: torch.from_numpy(v).to(DEV) for k, v in kw.items()}
    for lead, width in ((0, 3334), (1, 3400), (8, 3352), (3, 4001)):
        wide = torch.full((B, width), 1e4, dtype=dtype, device=DEV)
        wide[:, lead:lead + V] = x
        view = wide[:, lead:lead + V]
        got = fl.fl_logits_process(view, **dev)
        _logits_check(x, kw, got)
        _logits_check(x, kw, fl.fl_logits_process(view, **dev, need_logits=False))
        out = torch.full((B, width + 3), -7.0, dtype=torch.float32, device=DEV)
        _logits_check(x, kw, fl.fl_logits_process(view, **dev, out=out[:, 2:V + 2]))
        assert bool((out[:, :2] == -7).all()) and bool((out[:, V + 2:] == -7).all())
        if dtype == torch.float32:
            _logits_check(x, kw, fl.fl_logits_process(view, **dev, out=view))
            assert bool((wide[:, :lead] == 1e4).all()) and bool((wide[:, lead + V:] == 1e4).all())


def test_logits_repeats_and_graphs():
    x, kw = _logits_case(7, 128003, 3, torch.float32, history=300, biases=5)
    dev = {k: torch.from_numpy(v).to(DEV) for k, v in kw.items()}
    want = fl.fl_logits_process(x, **dev)
    for _ in range(4):
        got = fl.fl_logits_process(x, **dev)
        assert all(torch.equal(got[k], want[k]) for k in want)
    ws = torch.zeros(fl.fl_logits_process_workspace(7, 128003), dtype=torch.uint8, device=DEV)
    xin = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fl.fl_logits_process(xin, **dev, ws=ws)
    for _ in range(2):
        xin.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_offsets_past_32_bits():
    """Rows of the tokens, of y, of the logits and pages of a cache that lie more than 2^31 elements apart."""
    gap = 1500000000
    x, w, t = _linear_case(3, 300, 272, 2)
    want = fl.fl_int8_linear(x, w, t)
    far = torch.empty(2 * gap + 700, dtype=torch.bfloat16, device=DEV)
    xs, ys = far.as_strided((3, 272), (gap, 1)), far.as_strided((3, 300), (gap, 1), 300)
    xs.copy_(x)
    assert torch.equal(fl.fl_int8_linear(xs, w, t), want)
    fl.fl_int8_linear(x, w, t, y=ys)
    assert torch.equal(ys, want)
    lx, kw = _logits_case(3, 333, 1, torch.bfloat16, history=9)
    ls = far.as_strided((3, 333), (gap, 1))
    ls.copy_(lx)
    _logits_check(lx, kw, fl.fl_logits_process(ls, **{k: torch.from_numpy(v).to(DEV) for k, v in kw.items()}))
    del far, xs, ys, ls
    blocks = 70000                                   # of 64 KB of keys
    codes = [torch.zeros((blocks, 8, 64, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros((blocks, 8), device=DEV) for _ in range(2)]
    codes[0][blocks - 1], codes[1][2], scales[0][blocks - 1] = 7, 9, 3.0
    fl.fl_kv8_pages_copy(codes[:1], codes[1:], scales[:1], scales[1:], _i32([(blocks - 1, 1), (2, blocks - 2)]), _i32([2]))
    assert bool((codes[0][1] == 7).all()) and bool((codes[1][blocks - 2] == 9).all()) and bool((scales[0][1] == 3).all())
    assert not codes[0][0].any() and not codes[0][blocks - 2].any()


def test_linear_from_several_streams_at_once():
    """Calls that overlap on the GPU, each stream with the workspace that is its own."""
    cases = [_linear_case(M, N, 1040, M) for M, N in ((1, 3000), (40, 2000), (300, 1500), (20, 5000))]
    want = [fl.fl_int8_linear(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        for s, c, g in zip(streams, cases, got):
            with torch.cuda.stream(s):
                g.append(fl.fl_int8_linear(*c))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, y) for y in g)


def test_weights_rounded_just_before():
    """A linear right behind the kernels that make its weights and its tokens."""
    rng = np.random.default_rng(3)
    dense, x = _bf16(rng.standard_normal((900, 512))).to(DEV), _bf16(rng.standard_normal((70, 512))).to(DEV)
    w, t = fl.fl_int8_quantize(dense)
    torch.cuda.synchronize()
    for rows in (x[:3], x):
        want = fl.fl_int8_linear(rows, w, t)
        codes, scale = fl.fl_int8_quantize(rows)
        for _ in range(5):
            torch.zeros_like(w)                      # (the allocator hands this memory to the next call)
            w2, t2 = fl.fl_int8_quantize(dense)
            assert torch.equal(fl.fl_int8_linear(rows, w2, t2), want)
            del w2
            torch.zeros_like(w)
            w3, t3 = fl.fl_int8_quantize(dense)
            assert torch.equal(fl.fl_int8_linear(codes, w3, t3, x_scale=scale), want)
            del w3


# ------------------------------------------------------------------- pages

class _Pair:
    """A pool on the GPU beside the oracle's."""

    def __init__(self, blocks, slots, most, block):
        self.o = O.Pool(blocks, slots, most, block)
        self.block = block
        self.ws = torch.zeros(fl.fl_kv8_pages_workspace(blocks, slots, most, block), dtype=torch.uint8, device=DEV)
        self.upload()

    def upload(self):
        self.args = [_i32(self.o.refs), _i32(self.o.table), _i32(self.o.lens)]

    def same(self):
        refs, table, lens = (t.cpu().tolist() for t in self.args)
        assert refs == self.o.refs and lens == self.o.lens
        for s, n in enumerate(lens):
            assert table[s][:self.o.pages(n)] == self.o.table[s][:self.o.pages(n)]

    def free(self, seqs, keep=None):
        fl.fl_kv8_pages_free(*self.args, _i32(seqs), self.block, keep=_i32(keep) if keep is not None else None, status=self.ws)
        self.o.free(seqs, keep)
        self.same()

    def fork(self, parents, children):
        fl.fl_kv8_pages_fork(*self.args, _i32(parents), _i32(children), self.block, status=self.ws)
        self.o.fork(parents, children)
        self.same()

    def alloc(self, seqs, new):
        granted, pairs, count = fl.fl_kv8_pages_alloc(*self.args, _i32(seqs), _i32(new), self.block, ws=self.ws)
        ok, moves = self.o.alloc(seqs, new)
        assert granted.cpu().tolist() == ok and int(count) == len(moves)
        assert pairs.cpu().tolist() == [list(m) for m in moves] + [[-1, -1]] * (len(seqs) - len(moves))
        self.same()
        return ok, moves

    def compact(self, in_place):
        table, refs, pairs, count, moved = fl.fl_kv8_pages_compact(*self.args, self.block, in_place=in_place, status=self.ws)
        moves, where = self.o.compact()
        assert int(count) == len(moves) and moved.cpu().tolist() == where
        assert pairs.cpu().tolist() == [list(m) for m in moves] + [[-1, -1]] * (len(self.o.refs) // 2 - len(moves))
        assert in_place == (table.data_ptr() == self.args[1].data_ptr())
        self.args[0], self.args[1] = refs, table
        self.same()

    def status(self):
        return fl.fl_int4g_status(self.ws)


@pytest.mark.parametrize("blocks,slots,most,block", [(1, 1, 1, 16), (7, 3, 4, 16), (40, 12, 9, 32), (300, 64, 30, 16), (9001, 200, 70, 64),
                                                     (20000, 1500, 40, 128)])
def test_pages_random_lives(blocks, slots, most, block):
    import random
    rng = random.Random(blocks * 3 + slots)
    p = _Pair(blocks, slots, most, block)
    for step in range(12 if blocks > 1000 else 40):
        order = rng.sample(range(slots), rng.randint(1, slots))
        what = rng.choice(["alloc", "alloc", "alloc", "free", "cut", "fork", "compact"])
        if what == "alloc":
            new = [rng.choice([0, 1, 1, 1, 2, 5, block, 3 * block]) for _ in order]
            new = [min(n, most * block - p.o.lens[s]) for n, s in zip(new, order)]
            p.alloc(order, new)
        elif what == "free":
            p.free(order[:1 + len(order) // 4])
        elif what == "cut":
            p.free(order, [rng.randint(0, most * block) for _ in order])
        elif what == "fork":
            empty = [s for s in order if p.o.lens[s] == 0]
            full = [s for s in range(slots) if p.o.lens[s]]
            if empty and full:
                p.fork([rng.choice(full) for _ in empty], empty)
        else:
            p.compact(rng.random() < 0.5)
    assert p.status() == 0


@pytest.mark.parametrize("blocks,slots,most,block,seed", [(13, 10, 6, 16, 1), (50, 40, 8, 32, 2), (420, 300, 12, 16, 3), (1900, 1400, 9, 64, 4)])
def test_pages_crowded(blocks, slots, most, block, seed):
    """Many forks in a small pool: pages to copy, grants denied, pages moved, each many times."""
    import random
    rng = random.Random(seed)
    p = _Pair(blocks, slots, most, block)
    denied = copied = moved = 0
    for step in range(25):
        full = [s for s in range(slots) if p.o.lens[s]]
        empty = [s for s in range(slots) if not p.o.lens[s]]
        rng.shuffle(empty)
        if full and empty:
            p.fork([rng.choice(full) for _ in empty[1:]], empty[1:])
        order = rng.sample(range(slots), slots)
        ok, moves = p.alloc(order, [min(rng.choice([0, 1, 1, 2, block // 2, block]), most * block - p.o.lens[s]) for s in order])
        denied += ok.count(0)
        copied += len(moves)
        p.free(rng.sample(range(slots), slots // 2), [rng.randint(0, most * block) for _ in range(slots // 2)])
        p.free(rng.sample(range(slots), slots // 3))
        before = list(p.o.refs)
        p.compact(step % 2 == 0)
        moved += before != p.o.refs
    assert p.status() == 0 and denied and copied > 20 and moved > 5


def test_pages_lists_that_name_what_is_not_there():
    p = _Pair(50, 6, 5, 16)
    p.alloc([0, 1, 2], [20, 33, 1])
    assert p.status() == 0
    p.alloc([3, 3, 9, -1, 0, 1], [5, 5, 5, 5, -2, 10 ** 9])        # only the first entry counts
    assert p.status() == 6 and p.status() == 0
    p.fork([0, 0, 2, 7, 1, 0], [4, 4, 1, 5, -1, 2])                # a child twice, children that are parents, no slots
    assert p.status() == 6
    p.free([0, 0, 1, 77], [17, 3, 33, 0])                           # a slot twice: the least counts
    assert p.status() == 6
    p.free([4, 4])
    assert p.status() == 0
    p.fork([5], [0])                                                # a child that is not empty
    assert p.status() == 6
    p.args[1][1, 1] = 4000                                          # a page that the pool has not
    fl.fl_kv8_pages_free(*p.args, _i32([1]), 16, status=p.ws)
    assert p.status() == 6 and int(p.args[2][1]) == 0


def test_pages_empty_lists():
    p = _Pair(20, 4, 3, 32)
    p.alloc([], [])
    p.free([])
    p.fork([], [])
    p.compact(True)
    assert p.status() == 0


def test_pages_shared_by_all_of_a_list_and_by_others():
    p = _Pair(30, 8, 4, 16)
    p.alloc([0], [20])
    p.fork([0, 0, 0], [1, 2, 3])
    assert p.alloc([1, 2], [1, 1])[1] and p.o.refs[p.o.table[0][1]] == 2      # others hold it still: both copy
    assert len(p.alloc([3, 0], [1, 1])[1]) == 1                              # the last keeps it
    p.alloc([0, 1, 2, 3], [12, 12, 0, 30])
    p.free([0, 1, 2, 3])
    assert not any(p.o.refs)


def test_pages_grants_stop_at_the_first_that_does_not_fit():
    p = _Pair(6, 5, 6, 16)
    assert p.alloc([0, 1, 2, 3], [32, 40, 32, 1])[0] == [1, 1, 0, 0]
    p.alloc([3], [1])
    assert p.alloc([0, 1], [1, 1])[0] == [0, 0]


def _caches(layers, blocks, heads, block, dim, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    shape = (blocks, heads, block, dim)
    codes = [torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8) for _ in range(2 * layers)]
    scales = [torch.rand(shape[:2], generator=g, device=DEV) for _ in range(2 * layers)]
    return codes, scales


@pytest.mark.parametrize("layers,heads,block,dim", [(1, 1, 16, 64), (3, 5, 32, 128), (2, 8, 64, 128), (1, 40, 128, 128), (70, 2, 16, 64)])
def test_pages_copy(layers, heads, block, dim):
    blocks = 23
    codes, scales = _caches(layers, blocks, heads, block, dim, layers)
    before = [t.clone() for t in codes + scales]
    pairs = [(3, 20), (4, 1), (22, 0), (-1, 5), (6, 23), (2, 19), (7, 8)]
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    fl.fl_kv8_pages_copy(codes[0::2], codes[1::2], scales[0::2], scales[1::2], _i32(pairs), _i32([6]), status=st)
    for t, old in zip(codes + scales, before):
        want = old.clone()
        for f, to in pairs[:6]:
            if 0 <= f < blocks and 0 <= to < blocks:
                want[to] = old[f]
        assert torch.equal(t, want)
    assert fl.fl_int4g_status(st) == 6
    for n in (0, -4):
        now = [t.clone() for t in codes]
        fl.fl_kv8_pages_copy(codes[0::2], codes[1::2], scales[0::2], scales[1::2], _i32(pairs), _i32([n]), status=st)
        assert all(torch.equal(a, b) for a, b in zip(codes, now))
    fl.fl_kv8_pages_copy(codes[0::2], codes[1::2], scales[0::2], scales[1::2], _i32([(1, 2)]), _i32([100]), status=st)
    assert torch.equal(codes[-1][1], codes[-1][2]) and fl.fl_int4g_status(st) == 0
