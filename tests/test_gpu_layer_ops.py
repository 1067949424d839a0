"""GPU parity of the decoder-layer operators (RMS norm, rotary positions, the
8-bit cache's write and the attention over it) against the float64 oracle.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of f16
2^-11, of e4m3 2^-4; fp32 arithmetic adds terms of 2^-20 and less."""
import numpy as np
import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
FMT = {"e4m3": O.E4M3, "int8": O.INT8}


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


# ------------------------------------------------------------------ rmsnorm

def _norm_check(x, w, r, out, group, eps):
    s, n = O.rmsnorm(_np(x), _np(r) if r is not None else None, _np(w) if w is not None else None, eps)
    rel = 2.0 ** -18
    if "y" in out:
        assert np.all(np.abs(_np(out["y"]) - n) <= (2.0 ** -8 + rel) * np.abs(n) + 1e-38)
    if r is not None:
        assert np.all(np.abs(_np(out["residual"]) - s) <= (2.0 ** -8 + rel) * np.abs(s) + 1e-38)
    if "codes" in out:
        g = group or n.shape[-1]
        parts = n.reshape(*n.shape[:-1], -1, g)
        top = np.abs(parts).max(-1)
        scale = _np(out["scales"])
        assert scale.shape == top.shape
        assert np.all(np.abs(scale - top / 448) <= rel * top / 448 + 1e-38)
        got = O.values(out["codes"].cpu().numpy(), O.E4M3).reshape(parts.shape) * scale[..., None]
        # half a step: 2^-4 of a normal value, 2^-10 of the scale below
        assert np.all(np.abs(got - parts) <= (2.0 ** -4 + rel) * np.abs(parts) + (2.0 ** -10 + rel) * scale[..., None])


@pytest.mark.parametrize("H", [1, 7, 8, 64, 100, 256, 1000, 1024, 1032, 2048, 4096, 5000, 7168, 8192, 11008, 16384, 32768])
@pytest.mark.parametrize("M", [1, 3])
def test_rmsnorm_widths(H, M):
    rng = np.random.default_rng(H * 10 + M)
    x, r = _bf16(rng.standard_normal((M, H))).to(DEV), _bf16(3 * rng.standard_normal((M, H))).to(DEV)
    w = _bf16(1 + 0.3 * rng.standard_normal(H)).to(DEV)
    group = 128 if H % 128 == 0 else 0
    out = fl.fl_rmsnorm(x, w, 1e-5, residual=r, out8=True, group=group)
    _norm_check(x, w, r, out, group, 1e-5)
    out = fl.fl_rmsnorm(x, None, 1e-5)
    _norm_check(x, None, None, out, 0, 1e-5)


@pytest.mark.parametrize("H", [33, 300, 511, 700, 1030, 2046, 2816, 5001, 6144, 11003, 20001])
def test_rmsnorm_odd_widths(H):
    """Every number of vectors a thread, 16 bytes at a time and one by one."""
    rng = np.random.default_rng(H)
    x, r = _bf16(rng.standard_normal((5, H))).to(DEV), _bf16(2 * rng.standard_normal((5, H))).to(DEV)
    w = _bf16(1 + 0.2 * rng.standard_normal(H)).to(DEV)
    _norm_check(x, w, r, fl.fl_rmsnorm(x, w, 1e-6, residual=r, out8=True), 0, 1e-6)
    shifted = torch.zeros(5 * H + 1, dtype=torch.bfloat16, device=DEV)[1:].view(5, H)
    shifted.copy_(x)
    _norm_check(shifted, w, None, fl.fl_rmsnorm(shifted, w, 1e-6), 0, 1e-6)


@pytest.mark.parametrize("M", [2, 33, 700])
@pytest.mark.parametrize("group", [0, 64, 128, 256])
def test_rmsnorm_groups_and_rows(M, group):
    rng = np.random.default_rng(M + group)
    H = 768
    x = rng.standard_normal((M, H)) * 10.0 ** rng.integers(-4, 4, (M, 1))
    x[0, :256] = 0                                 # a run of zeros
    x, w = _bf16(x).to(DEV), _bf16(rng.standard_normal(H)).to(DEV)
    out = fl.fl_rmsnorm(x, w, 1e-6, out8=True, group=group, need_y=False)
    assert "y" not in out
    _norm_check(x, w, None, out, group, 1e-6)
    if group:
        assert float(out["scales"][0, 0]) == 0.0 and not out["codes"][0, :group].any()


@pytest.mark.parametrize("D", [64, 128, 80, 35])
def test_rmsnorm_heads_in_place(D):
    """Each query head of a wider projection normed by itself, where it lies."""
    rng = np.random.default_rng(D)
    qkv = _bf16(rng.standard_normal((9, 7, D))).to(DEV)
    w = _bf16(1 + 0.1 * rng.standard_normal(D)).to(DEV)
    before = qkv.clone()
    view = qkv[:, 2:6]
    out = fl.fl_rmsnorm(view, w, 1e-6, y=view)
    assert out["y"].data_ptr() == view.data_ptr()
    _norm_check(before[:, 2:6], w, None, {"y": view}, 0, 1e-6)
    assert torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 6:], before[:, 6:])


@pytest.mark.parametrize("H", [8, 24, 64, 72, 128])
@pytest.mark.parametrize("M,heads", [(1, 1), (5, 3), (37, 7), (600, 5)])
def test_rmsnorm_narrow_rows(M, heads, H):
    """Several rows a warp, with and without residual and weight; the last CTA
    partly filled, rows of a wider projection."""
    rng = np.random.default_rng(M + H)
    wide = _bf16(rng.standard_normal((M, heads + 2, H))).to(DEV)
    r = _bf16(3 * rng.standard_normal((M, heads, H))).to(DEV)
    w = _bf16(1 + 0.1 * rng.standard_normal(H)).to(DEV)
    x = wide[:, 1:1 + heads]
    _norm_check(x, w, r, fl.fl_rmsnorm(x, w, 1e-6, residual=r), 0, 1e-6)
    _norm_check(x, None, None, fl.fl_rmsnorm(x, None, 1e-5), 0, 1e-5)


def test_rmsnorm_residual_in_place_and_misaligned():
    rng = np.random.default_rng(3)
    buf = _bf16(rng.standard_normal((5, 264))).to(DEV)
    x = buf[:, 1:257]                              # rows off the 16-byte grid
    r = _bf16(rng.standard_normal((5, 256))).to(DEV)
    r0 = r.clone()
    out = fl.fl_rmsnorm(x, None, 1e-6, residual=r, residual_out=r, out8=True, group=64)
    _norm_check(x, None, r0, out, 64, 1e-6)
    # aligned rows give the same bits
    again = fl.fl_rmsnorm(x.contiguous(), None, 1e-6, residual=r0, out8=True, group=64)
    for k in ("y", "residual", "codes", "scales"):
        assert torch.equal(out[k], again[k]), k


def test_rmsnorm_zero_row_and_nan():
    x = torch.zeros((3, 128), dtype=torch.bfloat16, device=DEV)
    x[1] = 1.0
    x[2, 5] = float("nan")
    y = fl.fl_rmsnorm(x, None, 0.0 + 1e-6)["y"]
    assert not y[0].any() and torch.allclose(y[1].float(), torch.ones(128, device=DEV)) and bool(y[2].isnan().all())


# --------------------------------------------------------------------- rope

def _rope_check(x, y, pos, f, axis, halves, rot):
    ref = O.rope(_np(x), pos, f, axis, halves)
    mag = np.abs(_np(x)).copy()
    n = rot // 2
    a, b = (slice(0, n), slice(n, rot)) if halves else (slice(0, rot, 2), slice(1, rot, 2))
    both = mag[..., a] + mag[..., b]
    mag[..., a], mag[..., b] = both, both
    # the angle's last bit is 2^-32 turns of 2^31, in fp32 2^-25 turns: 2e-7 rad
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -22 + 4e-7) * mag
    tol[..., rot:] = 0
    err = np.abs(_np(y) - ref)
    assert np.all(err <= tol), np.max(err - tol)


@pytest.mark.parametrize("halves", [True, False])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,sections", [
    (1, 1, 1, 64, 64, None), (1, 32, 8, 128, 128, None), (5, 3, 1, 128, 64, [16, 8, 8]), (37, 8, 2, 64, 64, [10, 22]),
    (3, 2, 2, 80, 20, [4, 3, 3]), (700, 1, 1, 128, 128, [16, 24, 24]), (2, 2, 1, 10, 6, None), (9, 5, 0, 128, 128, None),
    (4, 1, 1, 1024, 1024, [100, 200, 150, 62]), (2, 40, 8, 96, 96, [0, 48]),
])
def test_rope(halves, T, Hq, Hk, D, rot, sections):
    rng = np.random.default_rng(T * 1000 + D + rot)
    A = len(sections) if sections else 1
    q, k = _bf16(rng.standard_normal((T, Hq, D))).to(DEV), _bf16(rng.standard_normal((T, Hk, D))).to(DEV) if Hk else None
    pos = rng.integers(0, 5000, (A, T))
    f = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    axis = np.repeat(np.arange(A), sections if sections else [rot // 2])
    P, F = _i32(pos), torch.from_numpy(f).to(DEV)
    qo, ko = fl.fl_rope(q, k, P, F, sections=sections, halves=halves)
    _rope_check(q, qo, pos, f, axis, halves, rot)
    if Hk:
        _rope_check(k, ko, pos, f, axis, halves, rot)
    # in place gives the same bits, and the negated positions undo it
    qi, ki = q.clone(), k.clone() if Hk else None
    fl.fl_rope(qi, ki, P, F, sections=sections, halves=halves, q_out=qi, k_out=ki)
    assert torch.equal(qi, qo) and (not Hk or torch.equal(ki, ko))
    back, _ = fl.fl_rope(qo, None, -P, F, sections=sections, halves=halves)
    assert torch.allclose(back.float(), q.float(), atol=0.06, rtol=0.02)


def test_rope_far_and_negative_positions():
    """Angles of far positions are as exact as near ones."""
    rng = np.random.default_rng(0)
    pos = np.array([[0, 1, 131071, 1000003, -1, -77777, 2 ** 31 - 1, -2 ** 31]])
    q = _bf16(rng.standard_normal((8, 2, 128))).to(DEV)
    f = 500000.0 ** (-np.arange(64) / 64)
    y, _ = fl.fl_rope(q, None, _i32(pos), torch.from_numpy(f).to(DEV))
    _rope_check(q, y, pos, f, np.zeros(64, int), True, 128)


def test_rope_strided():
    """Queries and keys inside one fused projection, rotated where they lie."""
    rng = np.random.default_rng(2)
    qkv = _bf16(rng.standard_normal((11, 8, 64))).to(DEV)
    before = qkv.clone()
    f = 10000.0 ** (-np.arange(32) / 32)
    pos = np.arange(11)[None]
    q, k = qkv[:, :4], qkv[:, 4:6]
    fl.fl_rope(q, k, _i32(pos[0]), torch.from_numpy(f).to(DEV), q_out=q, k_out=k)
    _rope_check(before[:, :6], qkv[:, :6], pos, f, np.zeros(32, int), True, 64)
    assert torch.equal(qkv[:, 6:], before[:, 6:])


# -------------------------------------------------------------------- append

def _table(rng, lens, block, spare=2):
    need = [-(-n // block) for n in lens]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)   # unused entries name no block
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


class Cache:
    """A device cache, and the host's copy for the oracle."""

    def __init__(self, blocks, heads, block, dim, fmt, rng=None, scales=None):
        shape = (blocks, heads, block, dim)
        self.fmt, self.codes, self.scale, self.dev = fmt, [], [], []
        for i in range(2):
            if rng is None:
                c, s = np.full(shape, 0x7f, np.uint8), np.full(shape[:2], np.nan, np.float32)
            else:
                c = O.codes(np.clip(rng.standard_normal(shape) * (100 if fmt == O.E4M3 else 40), -440, 440), fmt)
                s = (2.0 ** rng.integers(-9, -6, shape[:2])).astype(np.float32) if scales is None else scales[i]
            self.codes.append(c)
            self.scale.append(s)
            self.dev += [torch.from_numpy(c.copy()).to(DEV), torch.from_numpy(s.copy()).to(DEV)]

    def args(self):
        return self.dev[0], self.dev[2], self.dev[1], self.dev[3]

    def equal_host(self):
        return all(np.array_equal(self.dev[2 * i].cpu().numpy(), self.codes[i]) for i in range(2)) and all(
            np.array_equal(self.dev[2 * i + 1].cpu().numpy(), self.scale[i], equal_nan=True) for i in range(2))


def _cu(q):
    return [0, *np.cumsum(q).tolist()]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,block,heads", [(64, 16, 1), (128, 64, 3), (64, 128, 2), (128, 32, 2), (128, 128, 1)])
def test_append_steps(fmt, dim, block, heads):
    """Prompts, then tokens one by one and in chunks: codes and scales equal the
    oracle's bit for bit, and nothing else is written."""
    rng = np.random.default_rng(dim + block + heads)
    steps = [([1, block - 1, 2 * block + 5, 0], 1.0), ([1, 1, 1, 1], 5.0), ([1, 0, 1, block], 0.01), ([3, 2 * block, 7, 1], 40.0)]
    total = np.sum([s[0] for s in steps], 0)
    table, blocks = _table(rng, total, block)
    c = Cache(blocks, heads, block, dim, FMT[fmt])
    lens = np.zeros(4, int)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    for q, size in steps:
        lens = lens + q
        T = sum(q)
        kv = [_bf16(rng.standard_normal((T, heads, dim)) * size * np.exp(rng.standard_normal((T, 1, 1)))) for _ in range(2)]
        fl.fl_kv8_append(kv[0].to(DEV), kv[1].to(DEV), *c.args(), _i32(table), _i32(lens), cu_q=_i32(_cu(q)),
                         max_q=max(q), fmt=FMT[fmt], status=st)
        for i in range(2):
            O.append(_np(kv[i]), c.codes[i], c.scale[i], table, lens, _cu(q), FMT[fmt])
        assert c.equal_host()
    assert fl.fl_int4g_status(st) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_uniform_strided_many(fmt):
    """300 sequences of one token each, keys and values inside one projection."""
    rng = np.random.default_rng(7)
    lens = rng.integers(1, 70, 300)
    table, blocks = _table(rng, lens, 32)
    c = Cache(blocks, 2, 32, 64, FMT[fmt], rng)
    x = _bf16(rng.standard_normal((300, 8, 64)))
    d = x.to(DEV)
    fl.fl_kv8_append(d[:, 4:6], d[:, 6:], *c.args(), _i32(table), _i32(lens), fmt=FMT[fmt])
    for i in range(2):
        O.append(_np(x[:, 4 + 2 * i:6 + 2 * i]), c.codes[i], c.scale[i], table, lens, list(range(301)), FMT[fmt])
    assert c.equal_host()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_values(fmt):
    """Zeros, subnormals, the largest values, infinities and NaN."""
    c = Cache(3, 1, 16, 64, FMT[fmt])
    x = torch.zeros((16 * 3, 1, 64), dtype=torch.bfloat16)
    x[16, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1.0])
    x[17, 0, 0] = 3e38
    x[32, 0, :3] = torch.tensor([1e-40, -2e-39, 3e-38])
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    fl.fl_kv8_append(x.to(DEV), -x.to(DEV), *c.args(), _i32([[2, 0, 1]]), _i32([48]), fmt=FMT[fmt], status=st)
    for i in range(2):
        O.append(_np(x) * (1 - 2 * i), c.codes[i], c.scale[i], [[2, 0, 1]], [48], [0, 48], FMT[fmt])
    assert c.equal_host()
    assert fl.fl_int4g_status(st) == 7 and fl.fl_int4g_status(st) == 0


def test_append_more_rows_than_tokens():
    """Rows of negative positions are left out."""
    rng = np.random.default_rng(1)
    c = Cache(2, 1, 16, 64, O.INT8, rng)
    x = _bf16(rng.standard_normal((6, 1, 64)))
    fl.fl_kv8_append(x.to(DEV), x.to(DEV), *c.args(), _i32([[1]]), _i32([4]), fmt=O.INT8)
    for i in range(2):
        O.append(_np(x), c.codes[i], c.scale[i], [[1]], [4], [0, 6], O.INT8)
    assert c.equal_host()


# ------------------------------------------------------------------ attention

def _attend(lens, Hq, Hk, dim, block, fmt, window=0, seed=0, scales=None, scale=None, uniform=False, mutate=None, qgain=1.0):
    """Attention on the device and the oracle's; lens: (rows, cached tokens)."""
    rng = np.random.default_rng(seed)
    q_len, kv = [a for a, _ in lens], [b for _, b in lens]
    table, blocks = _table(rng, kv, block)
    c = Cache(blocks, Hk, block, dim, FMT[fmt], rng, scales(rng, (blocks, Hk)) if scales else None)
    for b, n in enumerate(kv):   # slots past the end hold anything: NaN codes, the largest codes
        if n % block:
            for i in range(2):
                c.codes[i][table[b, n // block], :, n % block:] = 0x7f if i == 0 else 0xff
                c.dev[2 * i].copy_(torch.from_numpy(c.codes[i]))
    T = sum(q_len)
    q = _bf16(rng.standard_normal((T, Hq + 3, dim)) * qgain)
    if mutate:
        mutate(q)
    scale = dim ** -0.5 if scale is None else scale
    ws = torch.zeros(fl.fl_kv8_attention_workspace(T, len(lens), Hq, Hk, dim), dtype=torch.uint8, device=DEV)
    kw = {} if uniform else dict(cu_q=_i32(_cu(q_len)), max_q=max(max(q_len), 1))
    args = (q.to(DEV)[:, 1:1 + Hq], *c.args(), _i32(table), _i32(kv))
    out, lse = fl.fl_kv8_attention(*args, fmt=FMT[fmt], scale=scale, window=window, return_lse=True, ws=ws, **kw)
    again, lse2 = fl.fl_kv8_attention(*args, fmt=FMT[fmt], scale=scale, window=window, return_lse=True, ws=ws, **kw)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse.view(torch.int32), lse2.view(torch.int32))
    assert fl.fl_int4g_status(ws) == 0
    assert not ws[:262400].any()                   # the counters are zero again
    ref = O.attention(_np(q[:, 1:1 + Hq]), c.codes[0], c.codes[1], c.scale[0], c.scale[1], table, kv, _cu(q_len), FMT[fmt],
                      scale, window)
    return out, lse, ref


def _close(out, lse, ref):
    o, l, tol, ltol = ref
    got, gl = _np(out), _np(lse)
    assert np.array_equal(np.isneginf(gl), np.isneginf(l))
    err = np.abs(got - o)
    assert np.all(err <= tol), (np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))
    f = np.isfinite(l)
    assert np.all(np.abs(gl[f] - l[f]) <= ltol[f]), np.max(np.abs(gl[f] - l[f]) / ltol[f])


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_attention_single_tokens(fmt, dim, block):
    """One row a sequence, every length around the tiles' and blocks' ends."""
    _close(*_attend([(1, n) for n in EDGES], 8, 2, dim, block, fmt, seed=dim + block, uniform=True))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 12, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_groups(group, dim):
    _close(*_attend([(1, 200), (2, 130), (0, 50), (3, 3), (1, 1)], 2 * group, 2, dim, 32, "e4m3", seed=group))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 6])
def test_attention_chunks(fmt, dim, group):
    """Several rows a sequence, after a context and from the start, rows
    without a token, sequences without rows."""
    _close(*_attend([(40, 40), (9, 170), (33, 300), (0, 10), (5, 2), (4, 0), (1, 129)], group, 1, dim, 16, fmt, seed=group))


@pytest.mark.parametrize("n", [63, 64, 65, 127, 128, 129, 200, 257])
def test_attention_prompts(n):
    """Whole prompts around the ends of row tiles."""
    _close(*_attend([(n, n)], 2, 1, 128, 64, "e4m3", seed=n))
    _close(*_attend([(n, n + 77), (1, 40)], 2, 2, 64, 16, "int8", seed=n))


@pytest.mark.parametrize("window", [1, 5, 16, 100, 128, 1000])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_window(window, dim):
    _close(*_attend([(1, 400), (7, 300), (1, 3), (150, 290), (2, 129)], 4, 2, dim, 16, "e4m3", window=window, seed=window))


def test_attention_window_leaves_freed_blocks_alone():
    """Blocks wholly before the window need not exist."""
    rng = np.random.default_rng(0)
    c = Cache(5, 1, 16, 64, O.INT8, rng)
    q = _bf16(rng.standard_normal((2, 2, 64)))
    table = np.array([[-1, -1, 3, 1, 4]], np.int32)
    ws = torch.zeros(fl.fl_kv8_attention_workspace(2, 1, 2, 1, 64), dtype=torch.uint8, device=DEV)
    out, lse = fl.fl_kv8_attention(q.to(DEV), *c.args(), _i32(table), _i32([75]), fmt=O.INT8, window=30, return_lse=True,
                                   ws=ws)
    assert fl.fl_int4g_status(ws) == 0
    full = np.array([[0, 0, 3, 1, 4]])
    _close(out, lse, O.attention(_np(q), *c.codes, *c.scale, full, [75], [0, 2], O.INT8, 0.125, 30))


@pytest.mark.parametrize("rows", [1, 150])
def test_attention_scales_far_apart(rows):
    """Scales over 2^24, blocks of zeros, large and small scores."""
    def scales(rng, shape):
        return [(2.0 ** rng.integers(-12, 12, shape)).astype(np.float32), (2.0 ** rng.integers(-14, 10, shape)).astype(np.float32)]
    _close(*_attend([(rows, 500), (rows, 350)], 4, 2, 128, 16, "e4m3", seed=5, scales=scales, scale=1e-3))

    def zeros(rng, shape):
        s = (2.0 ** rng.integers(-8, -6, shape)).astype(np.float32)
        s[::2] = 2.0 ** -126
        return [s, s.copy()]
    _close(*_attend([(rows, 500), (rows, 20)], 4, 2, 64, 16, "int8", seed=6, scales=zeros))
    # any positive scale, powers of two or not
    _close(*_attend([(rows, 200)], 4, 2, 64, 32, "int8", seed=7,
                    scales=lambda rng, shape: [rng.uniform(0.001, 0.02, shape).astype(np.float32) for _ in range(2)]))


@pytest.mark.parametrize("rows", [1, 150])
def test_attention_peaked_and_negative_scale(rows):
    _close(*_attend([(rows, 300)], 4, 2, 128, 64, "e4m3", seed=8, scale=3.0, qgain=4.0))
    _close(*_attend([(rows, 300)], 4, 2, 64, 64, "int8", seed=9, scale=-0.2))
    _close(*_attend([(rows, 300)], 4, 2, 64, 64, "int8", seed=9, scale=0.0))


@pytest.mark.parametrize("rows", [1, 150])
def test_attention_query_range(rows):
    """Queries outside f16's range, rows of zeros, a row with NaN."""
    def mutate(q):
        q[:] = (q.float() * 2.0 ** torch.randint(-60, 60, (q.shape[0], q.shape[1], 1)).float()).to(torch.bfloat16)
        q[0, 1] = 0
    out, lse, ref = _attend([(rows, 200), (rows, 160)], 2, 1, 64, 16, "e4m3", seed=10, scale=1e-18, mutate=mutate)
    _close(out, lse, ref)

    def nan(q):
        q[0, 1, 3] = float("nan")
    out, lse, ref = _attend([(rows, 200)], 3, 1, 64, 16, "e4m3", seed=11, mutate=nan)
    assert bool(out[0, 0].isnan().all()) and bool(lse[0, 0].isnan())
    o, l, tol, ltol = ref
    got = _np(out)
    got[0, 0], o[0, 0] = 0, 0
    tol[0, 0] = 1
    assert np.all(np.abs(got - o) <= tol)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_long_context(fmt):
    """Contexts over many CTAs' runs, next to short ones."""
    _close(*_attend([(1, 30000), (1, 5), (2, 9001)], 4, 1, 128, 64, fmt, seed=12))
    # a few rows more than the single-token form takes, over many CTAs
    _close(*_attend([(17, 20000)], 4, 1, 128, 64, fmt, seed=15))
    _close(*_attend([(3, 700), (70, 9000)], 2, 2, 64, 16, fmt, seed=16))


def test_attention_many_sequences():
    rng = np.random.default_rng(3)
    lens = [(int(rng.integers(0, 3)), int(n)) for n in rng.integers(0, 150, 620)]
    _close(*_attend(lens, 2, 1, 64, 16, "int8", seed=13))


def test_attention_mixed_rows():
    """Single tokens next to prompts in one call."""
    _close(*_attend([(1, 700), (130, 130), (1, 1), (70, 333), (3, 90), (1, 2000)], 4, 1, 128, 32, "e4m3", seed=14))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("mantissas", [False, True])
def test_attention_sequences_of_falling_length(fmt, mantissas):
    """A CTA's run goes from a long sequence's last tokens to a shorter one,
    and every page has a scale of its own."""
    def scales(rng, shape):
        return [(2.0 ** rng.integers(-11, -5, shape) * (rng.uniform(1, 2, shape) if mantissas else 1)).astype(np.float32)
                for _ in range(2)]
    _close(*_attend([(58, 226), (43, 126), (26, 240)], 4, 1, 128, 32, fmt, seed=17, scales=scales))
    _close(*_attend([(90, 2000), (70, 1500), (90, 1100), (40, 300), (33, 33)], 4, 2, 64, 16, fmt, seed=18, scales=scales))
    _close(*_attend([(300, 1900), (150, 700), (70, 100)], 3, 1, 64, 64, fmt, window=300, seed=19, scales=scales))


def test_attention_far_blocks():
    """Blocks whose codes lie more than 2^32 bytes into the cache."""
    rng = np.random.default_rng(4)
    blocks, heads, block, dim = 68000, 8, 64, 128
    dev = [torch.empty((blocks, heads, block, dim), dtype=torch.uint8, device=DEV) for _ in range(2)]
    small = Cache(8, heads, block, dim, O.E4M3, rng)
    ids = np.array([67999, 1, 65600, 67000, 3, 66001, 67998, 0])
    at = torch.from_numpy(ids).to(DEV)
    scale = [torch.ones((blocks, heads), dtype=torch.float32, device=DEV) for _ in range(2)]
    for i in range(2):
        dev[i][at] = small.dev[2 * i]
        scale[i][at] = small.dev[2 * i + 1]
    for rows in (1, 140):
        q = _bf16(rng.standard_normal((rows, 16, dim)))
        out, lse = fl.fl_kv8_attention(q.to(DEV), *dev, *scale, _i32(ids[None]), _i32([500]), return_lse=True)
        _close(out, lse, O.attention(_np(q), *small.codes, *small.scale, [list(range(8))], [500], [0, rows], O.E4M3, dim ** -0.5))
    # and the write there
    x = _bf16(rng.standard_normal((4, heads, dim)))
    fl.fl_kv8_append(x.to(DEV), x.to(DEV), *dev, *scale, _i32(ids[None]), _i32([68]))
    for i in range(2):
        O.append(_np(x), small.codes[i], small.scale[i], [list(range(8))], [68], [0, 4], O.E4M3)
        assert np.array_equal(dev[i][at].cpu().numpy(), small.codes[i])


@pytest.mark.parametrize("rows", [1, 150])
def test_attention_bad_blocks_are_reported(rows):
    """A block number outside the cache is not read: an error in the status
    block, other sequences right.  (What the kernels take from such a list is
    checked on the host.)"""
    rng = np.random.default_rng(5)
    c = Cache(20, 1, 16, 64, O.INT8, rng)
    table = np.stack([np.arange(10), np.arange(10, 20)]).astype(np.int32)
    table[0, 3] = 20
    q = _bf16(rng.standard_normal((2 * rows, 2, 64)))
    ws = torch.zeros(fl.fl_kv8_attention_workspace(2 * rows, 2, 2, 1, 64), dtype=torch.uint8, device=DEV)
    out, lse = fl.fl_kv8_attention(q.to(DEV), *c.args(), _i32(table), _i32([160, 160]), fmt=O.INT8, return_lse=True, ws=ws)
    assert fl.fl_int4g_status(ws) == 6
    o, l, tol, _ = O.attention(_np(q[rows:]), *c.codes, *c.scale, table[1:], [160], [0, rows], O.INT8, 0.125)
    assert np.all(np.abs(_np(out[rows:]) - o) <= tol)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    table[0, 9] = -7
    fl.fl_kv8_append(q[:, :1].to(DEV).contiguous(), q[:, 1:].to(DEV).contiguous(), *c.args(), _i32(table),
                     _i32([160, 160]), fmt=O.INT8, status=st)
    assert fl.fl_int4g_status(st) == 6


def test_append_then_attend():
    """A prompt and tokens after it through both, against attention over the
    unrounded keys and values: the 8-bit steps are all that differs."""
    rng = np.random.default_rng(6)
    for fmt, step in (("e4m3", 2.0 ** -4), ("int8", 2.0 ** -7)):
        c = Cache(12, 2, 16, 64, FMT[fmt])
        table, n = _i32([list(range(11, -1, -1))]), 0
        ks, vs = [], []
        for rows in (100, 1, 1, 7, 1):
            k, v, q = (_bf16(rng.standard_normal((rows, h, 64))) for h in (2, 2, 4))
            n += rows
            fl.fl_kv8_append(k.to(DEV), v.to(DEV), *c.args(), table, _i32([n]), fmt=FMT[fmt])
            out = fl.fl_kv8_attention(q.to(DEV), *c.args(), table, _i32([n]), fmt=FMT[fmt])
            ks.append(_np(k))
            vs.append(_np(v))
        k, v = np.concatenate(ks), np.concatenate(vs)
        for h in range(4):
            s = k[:, h // 2] @ _np(q)[0, h] / 8
            p = np.exp(s - s.max())
            p /= p.sum()
            ref = p @ v[:, h // 2]
            assert np.abs(_np(out)[0, h] - ref).max() < 4 * step      # |v| < 5, scores move by about a step


@pytest.mark.parametrize("rows", [1, 140])
def test_layer_ops_on_a_stream_and_in_a_graph(rows):
    """The operators on a stream of their own, then captured and replayed with
    other inputs and lengths."""
    rng = np.random.default_rng(8)
    s = torch.cuda.Stream()
    block, Hq, Hk, D, ctx = 32, 4, 2, 128, 90
    table = _i32([list(range(12)), list(range(12, 24))])
    x = torch.empty((2 * rows, Hq + 2 * Hk, D), dtype=torch.bfloat16, device=DEV)
    pos, lens = torch.empty(2 * rows, dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).to(DEV)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    c = Cache(24, Hk, block, D, O.E4M3, np.random.default_rng(1))
    start = [t.clone() for t in c.dev]
    ws = torch.zeros(fl.fl_kv8_attention_workspace(2 * rows, 2, Hq, Hk, D), dtype=torch.uint8, device=DEV)

    def step():
        n = fl.fl_rmsnorm(x[:, :Hq + Hk], w)["y"]
        q, k = fl.fl_rope(n[:, :Hq], n[:, Hq:], pos, f)
        fl.fl_kv8_append(k, x[:, Hq + Hk:], *c.args(), table, lens, status=ws)
        return fl.fl_kv8_attention(q, *c.args(), table, lens, ws=ws)

    def fill(seed, ctx):
        r = np.random.default_rng(seed)
        x.copy_(_bf16(r.standard_normal(tuple(x.shape))))
        lens.copy_(torch.tensor([ctx + rows, ctx // 2 + rows], dtype=torch.int32))
        pos.copy_(torch.cat([torch.arange(ctx, ctx + rows), torch.arange(ctx // 2, ctx // 2 + rows)]).int())
        for a, b in zip(c.dev, start):
            a.copy_(b)

    want = []
    for seed, n in ((1, ctx), (2, ctx + 60)):
        fill(seed, n)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            want.append(step())
        s.synchronize()
    g = torch.cuda.CUDAGraph()
    fill(1, ctx)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = step()
    for (seed, n), ref in zip(((1, ctx), (2, ctx + 60)), want):
        fill(seed, n)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
    assert fl.fl_int4g_status(ws) == 0
