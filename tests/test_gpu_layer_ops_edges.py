"""GPU parity of the decoder-layer operators at the edges of their arguments,
against the float64 oracle; tolerances as in test_gpu_layer_ops.py."""
import numpy as np
import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from oracle import layer_oracle as O
from test_gpu_layer_ops import DEV, FMT, Cache, _attend, _bf16, _close, _cu, _i32, _np, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from int4_group_quantized_int4g_gb300 import _build
    _build.build()
    fl.lib()


# ------------------------------------------------------------------ max_q

@pytest.mark.parametrize("dim,heads", [(128, 8), (64, 8), (128, 3)])
@pytest.mark.parametrize("lens", [[(4, 517)], [(1, 40)], [(1, 200), (1, 3), (2, 2), (0, 9)], [(1, 700)] * 8, [(40, 90), (1, 300)]])
def test_attention_loose_max_q(lens, dim, heads):
    """A bound larger than any sequence's rows, and than the call's: right
    results, and nothing behind the workspace is touched."""
    rng = np.random.default_rng(dim + len(lens))
    q_len, kv = [a for a, _ in lens], [b for _, b in lens]
    table, blocks = _table(rng, kv, 32)
    c = Cache(blocks, 1, 32, dim, O.E4M3, rng)
    T = sum(q_len)
    q = _bf16(rng.standard_normal((T, heads, dim)))
    ref = O.attention(_np(q), *c.codes, *c.scale, table, kv, _cu(q_len), O.E4M3, dim ** -0.5)
    need = fl.fl_kv8_attention_workspace(T, len(lens), heads, 1, dim)
    for max_q in (max(q_len), T, T + 1, 5, 16, 64, 4096, 2 ** 31 - 1):
        if max_q < max(q_len):
            continue
        # (64 MB behind the workspace, past what any of the kernels needs)
        room = torch.full((need + (64 << 20),), 0xa5, dtype=torch.uint8, device=DEV)
        room[:need] = 0
        out, lse = fl.fl_kv8_attention(q.to(DEV), *c.args(), _i32(table), _i32(kv), cu_q=_i32(_cu(q_len)), max_q=max_q,
                                       return_lse=True, ws=room[:need])
        _close(out, lse, ref)
        assert fl.fl_int4g_status(room[:need]) == 0
        assert bool((room[need:] == 0xa5).all()), max_q


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_loose_max_q(fmt):
    rng = np.random.default_rng(21)
    q_len, lens = [3, 0, 20, 1], [40, 5, 20, 33]
    table, blocks = _table(rng, lens, 16)
    x = _bf16(rng.standard_normal((24, 2, 64)))
    for max_q in (20, 24, 25, 4096, 2 ** 31 - 1):
        c = Cache(blocks, 2, 16, 64, FMT[fmt], np.random.default_rng(1))
        st = torch.zeros(4, dtype=torch.int32, device=DEV)
        fl.fl_kv8_append(x.to(DEV), -x.to(DEV), *c.args(), _i32(table), _i32(lens), cu_q=_i32(_cu(q_len)), max_q=max_q,
                         fmt=FMT[fmt], status=st)
        for i in range(2):
            O.append(_np(x) * (1 - 2 * i), c.codes[i], c.scale[i], table, lens, _cu(q_len), FMT[fmt])
        assert c.equal_host() and fl.fl_int4g_status(st) == 0


# ------------------------------------------------------------------ norm

def _small_runs_check(n, out, group):
    """Codes of runs down to fp32's last numbers: n to 2^-18 and a last place,
    the scale rounded to a last place (half of one, 2^-150, moves the 448
    steps of the largest code), half a step of e4m3 then."""
    g = group or n.shape[-1]
    parts = n.reshape(*n.shape[:-1], -1, g)
    top, rel, last = np.abs(parts).max(-1), 2.0 ** -18, 2.0 ** -149
    scale = _np(out["scales"])
    assert np.all(np.abs(scale - top / 448) <= rel * top / 448 + last)
    got = O.values(out["codes"].cpu().numpy(), O.E4M3).reshape(parts.shape)
    assert not np.isnan(got).any()
    assert not got[parts == 0].any()
    err = np.abs(got * scale[..., None] - parts)
    assert np.all(err <= (2.0 ** -4 + rel) * np.abs(parts) + (2.0 ** -10 + rel) * scale[..., None] + 449 * last)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("group", [0, 64, 128, 256])
def test_rmsnorm_codes_of_tiny_runs(group, aligned):
    """Runs of 1e-35 to 1e-40, with zeros among them: as columns of an otherwise
    normal row, by tiny weights, and as whole rows."""
    rng = np.random.default_rng(group + aligned)
    H, sizes = 1024, 10.0 ** -np.array([0.0, 36, 40, 35.5, 37, 38, 39, 36.3])
    x = rng.standard_normal((9, H))
    x[:, ::7] = 0
    gain = np.repeat(sizes, H // 8)                      # runs of 128 columns, of 256 with a larger half
    x[:4] *= gain
    x[4:6] *= 10.0 ** -np.array([[39.0], [40.0]])        # a whole row: n is 1000 times as large
    x[6, :] *= np.repeat(sizes[[1, 2]], H // 2)
    w = np.ones(H)
    w[256:512] = 1e-37
    buf = torch.zeros(9 * H + 8, dtype=torch.bfloat16, device=DEV)
    xd = (buf[:9 * H] if aligned else buf[1:9 * H + 1]).view(9, H)
    xd.copy_(_bf16(x))
    wd = _bf16(w).to(DEV)
    for weight in (None, wd):
        out = fl.fl_rmsnorm(xd, weight, 1e-6, out8=True, group=group)
        _, n = O.rmsnorm(_np(xd), None, _np(weight) if weight is not None else None, 1e-6)
        _small_runs_check(n, out, group)


def _shifted(x, aligned):
    """x on the device, on the 16-byte grid or one element off it."""
    buf = torch.zeros(x.numel() + 8, dtype=torch.bfloat16, device=DEV)
    d = buf[0 if aligned else 1:][:x.numel()].view(x.shape)
    d.copy_(x)
    return d


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("H", [8, 64, 128, 256, 1000, 1024, 3000, 4096, 8192, 16384, 32768])
def test_rmsnorm_rows_of_any_size(H, aligned):
    """Finite rows whose squares pass fp32, rows of tiny values without eps, and
    ordinary rows between them (neighbours of one warp in narrow rows)."""
    rng = np.random.default_rng(H + aligned)
    for sizes, eps in (([1.0, 1e19, 1e30, 1e38, 1e18, 1.0, 3e38, 1e25], 1e-6), ([1.0, 1e-16, 1e-20, 1e-30, 1e-39, 1.0, 1e-25, 1e38], 0.0),
                       ([1e-22, 1.0, 1e-18, 1e25], 1e-38)):
        x = rng.uniform(0.5, 1.0, (len(sizes), H)) * rng.choice([-1, 1], (len(sizes), H)) * np.array(sizes)[:, None]
        x = _shifted(_bf16(x), aligned)
        w = _shifted(_bf16(1 + 0.2 * rng.standard_normal(H)), aligned)
        r = _shifted(_bf16(0.1 * x.double().cpu().numpy() * rng.uniform(-1, 1, x.shape)), aligned)
        for weight, res in ((None, None), (w, r)):
            for out8 in (False, True):
                out = fl.fl_rmsnorm(x, weight, eps, residual=res, out8=out8)
                s = _np(x) + (_np(res) if res is not None else 0)
                n = s / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps) * (_np(w) if weight is not None else 1)
                assert np.all(np.abs(_np(out["y"]) - n) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(n) + 2.0 ** -133)
                if res is not None:   # (fp32 adds, then bf16: 2^-8 and 2^-24, subnormals to half their step)
                    assert np.all(np.abs(_np(out["residual"]) - s) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(s) + 2.0 ** -134)
                if out8:
                    _small_runs_check(n, out, 0)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("H", [8, 64, 128, 256, 1024, 4096, 16384])
def test_rmsnorm_infinities_and_nan(H, aligned):
    """A row with an infinity or a NaN gives NaN, all of it; the rows beside it
    are not touched by it."""
    rng = np.random.default_rng(H)
    x = rng.standard_normal((6, H))
    x[1, H // 2], x[2, 0], x[4, H - 1] = np.inf, -np.inf, np.nan
    xd, r = _shifted(_bf16(x), aligned), _shifted(_bf16(np.zeros((6, H))), aligned)
    for out8 in (False, True):
        out = fl.fl_rmsnorm(xd, None, 1e-6, residual=r, out8=out8, group=64 if H % 64 == 0 and out8 else 0)
        good = torch.tensor([True, False, False, True, False, True], device=DEV)
        assert bool(out["y"][~good].isnan().all())
        assert torch.equal(out["residual"].view(torch.int16), xd.view(torch.int16)) or bool(out["residual"][4, H - 1].isnan())
        _, n = O.rmsnorm(_np(xd[good]), None, None, 1e-6)
        assert np.all(np.abs(_np(out["y"][good]) - n) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(n))
        if out8:
            codes = O.values(out["codes"].cpu().numpy(), O.E4M3)
            g = good.cpu().numpy()
            assert np.isnan(codes[~g]).all() and not np.isnan(codes[g]).any()
            assert not out["scales"][~good].any()


# ------------------------------------------------------------------ attention, scores of any size

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,kv", [(1, 300), (1, 9000), (6, 700), (70, 300), (70, 9000)])
@pytest.mark.parametrize("size", [-1e33, -1e31, -3e29, -2.0 ** 27, 2.0 ** 27, 2.0 ** 29, 1e31])
def test_attention_equal_scores_of_any_size(size, rows, kv, fmt):
    """Equal keys: whatever the size of their score, the weights are equal.  (In
    log2 units scores reach 1e33 * 64 * 2.)"""
    rng = np.random.default_rng(rows + kv)
    block, dim, heads = 64, 64, 4
    blocks = -(-kv // block)
    c = Cache(blocks, 1, block, dim, FMT[fmt], rng)
    one = O.codes(np.full(dim, 96.0) + np.arange(dim) % 8, FMT[fmt])      # 1.5 and a little more, at 2^-6
    c.codes[0][:] = one
    c.scale[0][:] = 2.0 ** -6
    c.scale[1][:] = 2.0 ** -7
    for i in range(2):
        c.dev[2 * i].copy_(torch.from_numpy(c.codes[i]))
        c.dev[2 * i + 1].copy_(torch.from_numpy(c.scale[i]))
    q = _bf16(rng.uniform(0.9, 1.1, (rows, heads, dim)))
    s = size * (_np(q) @ (O.values(one, FMT[fmt]) * 2.0 ** -6))             # [rows, heads]
    ws = torch.zeros(fl.fl_kv8_attention_workspace(rows, 1, heads, 1, dim), dtype=torch.uint8, device=DEV)
    out, lse = fl.fl_kv8_attention(q.to(DEV), *c.args(), _i32(np.arange(blocks)[None]), _i32([kv]), fmt=FMT[fmt], scale=size,
                                   return_lse=True, ws=ws)
    v = O.gather(c.codes[1], c.scale[1], np.arange(blocks), kv, FMT[fmt])[0]
    got, gl = _np(out), _np(lse)
    for i in range(rows):
        n = kv - rows + 1 + i
        mean, av = v[:n].mean(0), np.abs(v[:n]).mean(0)
        # the output's rounding, the weights' to f16, the sums' (as in the oracle's tolerance, with exact scores)
        assert np.all(np.abs(got[i] - mean) <= 2.0 ** -8 * np.abs(mean) + (2.0 ** -11 + 2.0 ** -18) * av), (i, got[i, 0, :4], mean[:4])
        assert np.all(np.abs(gl[i] - s[i] - np.log(n)) <= (dim + 4) * 2.0 ** -23 * np.abs(s[i]) + 2.0 ** -20)
    assert fl.fl_int4g_status(ws) == 0


@pytest.mark.parametrize("rows", [1, 7, 90])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("log2", [16, 20, 22, 23, 24, 25, 26, 27, 28, 30, 40])
def test_attention_large_scores(log2, fmt, rows):
    """Scores that fp32 holds to whole numbers and coarser: outputs stay within
    what that rounding allows, mantissas in the scales or not."""
    for i, mantissas in enumerate((False, True)):
        def scales(rng, shape):
            return [(2.0 ** rng.integers(-9, -7, shape) * (rng.uniform(1, 2, shape) if mantissas else 1)).astype(np.float32)
                    for _ in range(2)]
        out, lse, ref = _attend([(rows, 400), (rows, 131)], 4, 2, 128, 32, fmt, seed=log2 + i, scales=scales,
                                scale=2.0 ** log2 * (1.3 if i else 1.0))
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
        _close(out, lse, ref)


# ------------------------------------------------------------------ lists

@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("bad", ["length", "falls", "rows", "past"])
def test_sequences_that_are_left_out_are_reported(bad, many):
    """A sequence whose lists name what is not there: an error in the status
    block, nothing written for it, the others right.  (What the kernels take from
    such lists is checked on the host.)"""
    rng = np.random.default_rng(7)
    n = 40 if many else 2                                              # rows: either attention kernel
    B, block = 300 if bad == "length" and not many else 3, 16
    q_len, kv = [n] * B, [int(k) for k in rng.integers(n, 60, B)]
    at = B - 1                                                         # the sequence that is left out
    table, blocks = _table(rng, kv, block)
    lens, cu, T, max_q = list(kv), _cu(q_len), B * n, n
    if bad == "length":
        lens[at] = table.shape[1] * block + 1
    elif bad == "falls":
        cu[at + 1] = cu[at] - 1
    elif bad == "past":
        cu[at + 1] = T + 1
    else:
        q_len[0], max_q = n - 1, n - 1                                 # (the others have as many rows as allowed)
        q_len[1], cu = n - 1, _cu([n - 1, n - 1, n])
    good = [b for b in range(B) if b != at]
    x = _bf16(rng.standard_normal((T, 2, 64)))
    c = Cache(blocks, 1, block, 64, O.E4M3, rng)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    fl.fl_kv8_append(x[:, :1].contiguous().to(DEV), x[:, 1:].contiguous().to(DEV), *c.args(), _i32(table), _i32(lens), cu_q=_i32(cu),
                     max_q=max_q, status=st)
    assert fl.fl_int4g_status(st) == 6
    for i in range(2):
        for b in good:
            O.append(_np(x[cu[b]:cu[b + 1], i:i + 1]), c.codes[i], c.scale[i], table[b:b + 1], [lens[b]], [0, cu[b + 1] - cu[b]], O.E4M3)
    assert c.equal_host()
    ws = torch.zeros(fl.fl_kv8_attention_workspace(T, B, 2, 1, 64), dtype=torch.uint8, device=DEV)
    out = torch.full((T, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    _, lse = fl.fl_kv8_attention(x.to(DEV), *c.args(), _i32(table), _i32(lens), cu_q=_i32(cu), max_q=max_q, out=out, return_lse=True, ws=ws)
    assert fl.fl_int4g_status(ws) == 6
    for b in good:
        rows = slice(cu[b], cu[b + 1])
        _close(out[rows], lse[rows], O.attention(_np(x[rows]), *c.codes, *c.scale, table[b:b + 1], [lens[b]], [0, cu[b + 1] - cu[b]], O.E4M3, 0.125))
    assert bool((out[cu[at - 1 if bad == "falls" else at] + (n if bad == "falls" else 0):] == 7.0).all())


def test_rows_of_no_sequence_are_left_alone():
    """Rows before the first sequence's and past the last's, as a padded batch
    has them, without an error; sequences without rows may have any length."""
    rng = np.random.default_rng(9)
    cu, kv = [2, 3, 3, 5], [40, 1 << 20, 17]
    table = np.array([[0, 1, 2], [-1, -1, -1], [3, 4, -1]], np.int32)
    c = Cache(5, 1, 16, 64, O.INT8, rng)
    x = _bf16(rng.standard_normal((8, 2, 64)))
    ws = torch.zeros(fl.fl_kv8_attention_workspace(8, 3, 2, 1, 64), dtype=torch.uint8, device=DEV)
    out = torch.full((8, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    fl.fl_kv8_append(x[:, :1].contiguous().to(DEV), x[:, 1:].contiguous().to(DEV), *c.args(), _i32(table), _i32(kv), cu_q=_i32(cu),
                     max_q=4, fmt=O.INT8, status=ws)
    for i in range(2):
        for b in (0, 2):
            O.append(_np(x[cu[b]:cu[b + 1], i:i + 1]), c.codes[i], c.scale[i], table[b:b + 1], [kv[b]], [0, cu[b + 1] - cu[b]], O.INT8)
    assert c.equal_host()
    _, lse = fl.fl_kv8_attention(x.to(DEV), *c.args(), _i32(table), _i32(kv), cu_q=_i32(cu), max_q=4, fmt=O.INT8, out=out,
                                 return_lse=True, ws=ws)
    assert fl.fl_int4g_status(ws) == 0
    for b in (0, 2):
        rows = slice(cu[b], cu[b + 1])
        _close(out[rows], lse[rows], O.attention(_np(x[rows]), *c.codes, *c.scale, table[b:b + 1], [kv[b]], [0, cu[b + 1] - cu[b]], O.INT8, 0.125))
    assert bool((out[:2] == 7.0).all()) and bool((out[5:] == 7.0).all())


# ------------------------------------------------------------------ workspaces of captured calls

@pytest.mark.parametrize("rows", [1, 40])
def test_captured_calls_without_a_workspace(rows):
    """Two graphs captured on one stream, the second replayed alone; then a larger
    call on that stream, and the first graph: partials are counted from zero in
    all of them."""
    rng = np.random.default_rng(12)
    kv = 3000
    c = Cache(-(-kv // 32), 1, 32, 128, O.E4M3, rng)
    table, lens = _i32(np.arange(-(-kv // 32))[None]), _i32([kv])
    q = _bf16(rng.standard_normal((rows, 4, 128))).to(DEV)
    big = torch.zeros((2 * rows + 300, 8, 128), dtype=torch.bfloat16, device=DEV)
    ref = O.attention(_np(q), *c.codes, *c.scale, [np.arange(-(-kv // 32))], [kv], [0, rows], O.E4M3, 128 ** -0.5)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for warm in (False, True):
        graphs = []
        for _ in range(2):
            if warm:
                with torch.cuda.stream(s):
                    fl.fl_kv8_attention(q, *c.args(), table, lens)
                s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out, lse = fl.fl_kv8_attention(q, *c.args(), table, lens, return_lse=True)
            graphs.append((g, out, lse))
        for i in (1, 0, 1):
            graphs[i][1].zero_()
            graphs[i][0].replay()
            torch.cuda.synchronize()
            _close(graphs[i][1], graphs[i][2], ref)
            with torch.cuda.stream(s):   # outgrows the stream's workspace, and takes what is free
                fl.fl_kv8_attention(big, *c.args(), table, lens)
                junk = [torch.full((1 << 22,), 0x5a, dtype=torch.uint8, device=DEV) for _ in range(8)]
            torch.cuda.synchronize()
        del junk


# ------------------------------------------------------------------ write, then read

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 64)])
@pytest.mark.parametrize("signs", [True, False])
def test_append_then_attend_every_row(signs, dim, block, fmt):
    """Prompts, chunks and single tokens through the write and the attention,
    every row of every step against attention over the unrounded keys and
    values.  Each query points at one token of its own choice, so that a token
    out of place or a wrong scale shows; with keys of signs alone, which either
    format holds as they are, to the rounding of a value.  Bounds: a code is off by half a step
    (e4m3 2^-4 of it, 2^-10 of the scale below; int8 1/2 of the scale) and by as
    much again of every smaller scale that its block had, which at least
    double: twice that part in all."""
    rng = np.random.default_rng(dim)
    heads, B = 4, 2
    steps = [([70, 33], 1.0), ([1, 1], 4.0), ([9, 40], 0.3), ([1, 1], 1.0), ([50, 2], 6.0), ([1, 1], 0.1)]
    total = np.sum([a for a, _ in steps], 0)
    table, blocks = _table(rng, total, block)
    c = Cache(blocks, 2, block, dim, FMT[fmt])
    lens, ks, vs = np.zeros(B, int), [np.zeros((0, 2, dim))] * B, [np.zeros((0, 2, dim))] * B

    def off(x):   # bound of a code's error, [tokens, heads, dim]
        e = np.zeros_like(x)
        for j in range(0, len(x), block):
            for h in range(2):
                s = O.least_scale(np.abs(x[j:j + block, h]).max(), FMT[fmt])
                e[j:j + block, h] = 2.0 ** -4 * np.abs(x[j:j + block, h]) + 2 * 2.0 ** -10 * s if fmt == "e4m3" else s
        return e
    for q_len, size in steps:
        new = [[_bf16(rng.choice([-1.0, 1.0], (n, 2, dim)) if signs and not i else
                      rng.standard_normal((n, 2, dim)) * (1 + rng.random((n, 1, 1))) * (size if i else 1)) for i in range(2)] for n in q_len]
        lens = lens + q_len
        for b in range(B):
            ks[b], vs[b] = np.concatenate([ks[b], _np(new[b][0])]), np.concatenate([vs[b], _np(new[b][1])])
        q = []
        for b in range(B):
            n = q_len[b]
            aim = [int(rng.integers(0, lens[b] - n + i + 1)) if i % 3 else lens[b] - n + i for i in range(n)]
            q.append(np.stack([3.0 * 64 / dim * ks[b][a][[0, 0, 1, 1]] for a in aim]))
        q = _bf16(np.concatenate(q))
        fl.fl_kv8_append(torch.cat([x[0] for x in new]).to(DEV), torch.cat([x[1] for x in new]).to(DEV), *c.args(), _i32(table),
                         _i32(lens), cu_q=_i32(_cu(q_len)), max_q=max(q_len), fmt=FMT[fmt])
        got = _np(fl.fl_kv8_attention(q.to(DEV), *c.args(), _i32(table), _i32(lens), cu_q=_i32(_cu(q_len)), max_q=max(q_len), fmt=FMT[fmt]))
        at = 0
        for b in range(B):
            dk, dv = off(ks[b]) * (not signs), off(vs[b])
            for i in range(q_len[b]):
                n = lens[b] - q_len[b] + i + 1
                for h in range(heads):
                    x, g = _np(q[at, h]), h // 2
                    s = ks[b][:n, g] @ x / dim ** 0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    v = vs[b][:n, g]
                    out = p @ v
                    more = np.exp(2 * (dk[:n, g] @ np.abs(x)).max() / dim ** 0.5)      # a weight's factor, at most
                    tol = (more * (p @ dv[:n, g]) + (more - 1) * (p @ np.abs(v - out)) + 2.0 ** -8 * np.abs(out)
                           + 2.0 ** -10 * (p @ np.abs(v)))
                    assert np.all(np.abs(got[at, h] - out) <= tol), (b, i, h, np.max(np.abs(got[at, h] - out) / tol))
                at += 1
