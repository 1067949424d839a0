"""Host side of the decoder-layer operators: refusals before any launch, what
the cache kernels make of malformed lists (the same code, run on the host),
and pins of their oracle.  No GPU."""
import ctypes
import random

import numpy as np
import pytest

import int4_group_quantized_int4g_gb300 as fl
from int4_group_quantized_int4g_gb300 import _build
from oracle import layer_oracle as O

A = ctypes.c_void_p(0x10000)       # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)
BYTE = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fl.lib()


def test_rmsnorm_refusals(L):
    def call(x=A, xs=256, r=None, rs=0, w=A, eps=1e-6, M=2, heads=1, H=256, y=A, ys=256, ro=None, ros=0, c=None, sc=None,
             group=0):
        return L.fl_rmsnorm(x, xs, r, rs, w, eps, M, heads, H, y, ys, ro, ros, c, sc, group, None)
    assert call(x=None) == 1
    assert call(y=None) == 1                          # nothing to write
    assert call(c=A) == 1 and call(sc=A) == 1         # codes and scales go together
    assert call(M=0) == 1 and call(heads=0) == 1 and call(H=0) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(xs=255) == 1 and call(ys=255) == 1
    assert call(r=A, rs=10) == 1 and call(ro=A, ros=10) == 1
    assert call(x=BYTE) == 1 and call(w=BYTE) == 1
    assert call(group=64) == 1                        # a group without codes
    assert call(c=A, sc=A, group=32) == 3
    assert call(c=A, sc=A, H=200, group=64) == 1
    assert call(H=32776, xs=40000, ys=40000) == 3


def test_rope_refusals(L):
    def call(q=A, qs=256, Hq=2, k=A, ks=128, Hk=1, T=3, D=128, rot=128, style=0, pos=A, axes=1, sec=None, f=A, qo=A,
             qos=256, ko=A, kos=128):
        s = (ctypes.c_int32 * len(sec))(*sec) if sec else None
        return L.fl_rope(q, qs, Hq, k, ks, Hk, T, D, rot, style, pos, axes, s, f, qo, qos, ko, kos, None)
    assert call(q=None) == 1 and call(k=None) == 1 and call(pos=None) == 1 and call(f=None) == 1
    assert call(qo=None) == 1 and call(ko=None) == 1
    assert call(T=0) == 1 and call(Hq=0) == 1 and call(Hk=-1) == 1
    assert call(rot=127) == 1 and call(rot=0) == 1 and call(rot=130) == 1
    assert call(style=2) == 1
    assert call(axes=0) == 1 and call(axes=5, sec=[16, 16, 16, 16, 0]) == 1
    assert call(axes=2) == 1                          # several axes need sections
    assert call(axes=2, sec=[32, 31]) == 1 and call(axes=2, sec=[65, -1]) == 1
    assert call(qs=255) == 1 and call(kos=127) == 1
    assert call(q=BYTE) == 1 and call(f=ctypes.c_void_p(0x10004)) == 1
    assert call(D=2048, qs=4096, qos=4096, ks=2048, kos=2048) == 3


def _cache(**kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, num_blocks=8, block=16, kv_heads=2, head_dim=64, format=0)
    d.update(kw)
    return fl.FlKv8Cache(**d)


def _seqs(**kw):
    d = dict(cu_q=A, kv_lens=A, block_table=A, T=4, B=2, max_q=2, max_blocks=4)
    d.update(kw)
    return fl.FlKv8Seqs(**d)


def test_cache_refusals(L):
    size = ctypes.c_size_t(0)
    assert L.fl_kv8_attention_workspace(4, 2, 4, 2, 64, ctypes.byref(size)) == 0 and size.value > 0
    assert L.fl_kv8_attention_workspace(4, 2, 3, 2, 64, ctypes.byref(size)) == 1
    assert L.fl_kv8_attention_workspace(4, 2, 4, 2, 80, ctypes.byref(size)) == 3

    def append(k=A, ks=128, v=A, vs=128, st=A, c=None, s=None):
        return L.fl_kv8_append(k, ks, v, vs, ctypes.byref(c or _cache()), ctypes.byref(s or _seqs()), st, None)

    def attend(q=A, qs=256, Hq=4, out=A, os=256, lse=None, ws=A, n=1 << 30, window=0, scale=0.1, c=None, s=None):
        return L.fl_kv8_attention(q, qs, Hq, ctypes.byref(c or _cache()), ctypes.byref(s or _seqs()), scale, window, out,
                                  os, lse, ws, n, None)
    for call in (append, attend):
        assert call(c=_cache(k=None)) == 1 and call(c=_cache(v_scale=None)) == 1 and call(c=_cache(v=ODD)) == 1
        assert call(c=_cache(k_scale=BYTE)) == 1 and call(s=_seqs(kv_lens=BYTE)) == 1
        assert call(c=_cache(num_blocks=0)) == 1 and call(c=_cache(kv_heads=0)) == 1 and call(c=_cache(format=2)) == 1
        for block in (0, 8, 48, 256):
            assert call(c=_cache(block=block)) == 3
        for dim in (32, 80, 256):
            assert call(c=_cache(head_dim=dim)) == 3
        assert call(c=_cache(num_blocks=1 << 27, block=128)) == 3            # more than 2^31 rows
        assert call(s=_seqs(kv_lens=None)) == 1 and call(s=_seqs(block_table=None)) == 1
        assert call(s=_seqs(T=0)) == 1 and call(s=_seqs(B=0)) == 1 and call(s=_seqs(max_q=0)) == 1
        assert call(s=_seqs(max_blocks=0)) == 1
        assert call(s=_seqs(cu_q=None, T=5)) == 1                            # T % B without a list
        assert call(s=_seqs(max_blocks=1 << 28)) == 3 and call(s=_seqs(T=1 << 30)) == 3
    assert append(k=None) == 1 and append(v=ODD) == 1 and append(st=None) == 1 and append(st=ODD) == 1
    assert append(ks=120) == 1 and append(vs=132) == 1
    assert attend(q=None) == 1 and attend(out=ODD) == 1 and attend(ws=None) == 1 and attend(lse=BYTE) == 1
    assert attend(Hq=3) == 1 and attend(Hq=0) == 1 and attend(window=-1) == 1
    assert attend(scale=float("nan")) == 1 and attend(scale=float("inf")) == 1
    assert attend(qs=248) == 1 and attend(os=260) == 1
    assert attend(n=1024) == 2


def test_wrappers_refuse():
    import torch
    with pytest.raises(ValueError):
        fl.fl_rmsnorm(torch.zeros(2, 8, dtype=torch.bfloat16))              # not on a GPU
    with pytest.raises(ValueError):
        fl.fl_kv8_append(*[torch.zeros(1, 2, 64, dtype=torch.bfloat16)] * 2, *[None] * 6)


def test_pages_of_well_formed_lists():
    table = [[3, 1, 4, 0], [7, 2, 5, 6]]
    r = fl.fl_kv8_test_pages([50, 33], table, 5, 8, 16, 0, cu_q=[0, 3, 5])
    assert (r["start"], r["rows"], r["kv"]) == (0, 3, 50)
    assert r["write"] == (2, 2, 0) and r["read"] == (0, 4, 0)               # tokens 47 .. 49; pages 0 .. 3
    r = fl.fl_kv8_test_pages([50, 33], table, 5, 8, 16, 1, cu_q=[0, 3, 5], window=4)
    assert (r["start"], r["rows"], r["kv"]) == (3, 2, 33)
    assert r["write"] == (1, 2, 0) and r["read"] == (1, 2, 0)               # the first row sees 28 .. 31
    r = fl.fl_kv8_test_pages([0], [[0]], 1, 8, 16, 0)                        # nothing cached
    assert r["kv"] == 0 and r["write"][1] == 0 and r["read"][1] == 0
    r = fl.fl_kv8_test_pages([2], [[0]], 5, 8, 16, 0)                        # fewer tokens than rows
    assert r["write"] == (0, 1, 0)


def test_pages_of_malformed_lists_stay_inside_the_arrays():
    rnd = random.Random(5)
    for _ in range(3000):
        B, T, block = rnd.randint(1, 4), rnd.randint(1, 40), rnd.choice([16, 32, 64, 128])
        mb, nb = rnd.randint(1, 5), rnd.randint(1, 6)
        big = [-2 ** 31, -1, 0, 1, 7, 16, 33, 100, 640, 2 ** 31 - 1]
        cu = [rnd.choice(big + list(range(T + 2))) for _ in range(B + 1)]
        lens = [rnd.choice(big) for _ in range(B)]
        table = [[rnd.choice([-2 ** 31, -1, nb, 2 ** 31 - 1, *range(nb)]) for _ in range(mb)] for _ in range(B)]
        window = rnd.choice([0, 1, 5, 100, 2 ** 31 - 1])
        max_q = rnd.randint(1, T)
        for b in range(B):
            r = fl.fl_kv8_test_pages(lens, table, T, nb, block, b, cu_q=cu, max_q=max_q, window=window)
            assert 0 <= r["start"] <= T and 0 <= r["rows"] <= max_q and r["start"] + r["rows"] <= T
            assert 0 <= r["kv"] <= mb * block
            for first, n, bad in (r["write"], r["read"]):
                assert first >= 0 and n >= 0 and (n == 0 or first + n <= mb)
                assert bad == sum(not 0 <= table[b][i] < nb for i in range(first, first + n))


def test_prompt_units_cover_every_visible_token():
    """Units of the attention of many rows against a count by hand: items in
    order, each tile with a visible token in exactly one unit, no more units
    than the causal triangle needs."""
    rnd = random.Random(9)
    for _ in range(400):
        group, window = rnd.choice([1, 2, 3, 5, 7, 8, 16]), rnd.choice([0, 0, 1, 64, 300, 1000, 10 ** 6])
        n = rnd.randint(1, 700)
        kv = max(0, n + rnd.choice([-n, -5, 0, 1, 127, 128, 1000, 5000]))
        items, units = fl.fl_kv8_test_units(n, kv, group, window=window)
        assert items == -(-n * group // 256)
        past, u = kv - n, 0
        for i in range(items):
            item, index, count, tile0, lim, low = fl.fl_kv8_test_units(n, kv, group, u, window)
            assert (item, index) == (i, 0)
            first, last = i * 256 // group, min(i * 256 + 255, n * group - 1) // group
            assert lim == past + last + 1 and low == (max(0, past + first + 1 - window) if window and window < kv else 0)
            assert tile0 == low // 128 and (tile0 + count) * 128 >= lim and count >= 1
            if past >= 0 and not (window and window < kv):
                assert count == -(-lim // 128)
            if count > 1:
                assert fl.fl_kv8_test_units(n, kv, group, u + count - 1, window)[:2] == (i, count - 1)
            u += count
        assert u == units


# ------------------------------------------------------------- oracle pins

def test_e4m3_rounding_pins():
    v = O.E4M3_VALUES
    ok = ~np.isnan(v)
    c = np.arange(256)[ok]
    assert np.array_equal(O.e4m3_codes(v[ok]), c)                            # every value is its own code
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and np.isnan(v[0x7f])
    # ties go to the even mantissa, larger magnitudes saturate
    assert list(O.e4m3_codes([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 1e9, -1e9])) == [0x38, 0x3a, 0, 2, 0x7e, 0xfe]


def test_scale_pins():
    assert O.least_scale(448.0, O.E4M3) == 1 and O.least_scale(449.0, O.E4M3) == 2 and O.least_scale(224.0, O.E4M3) == 0.5
    assert O.least_scale(127.0, O.INT8) == 1 and O.least_scale(127.5, O.INT8) == 2
    assert O.least_scale(0.0, O.INT8) == 2.0 ** -126 and O.least_scale(1e-45, O.E4M3) == 2.0 ** -126


def test_append_and_gather_pins():
    """On values that are codes at the scale, the cache returns them as they are."""
    x = np.array([[[1.0, -448.0] + [0.0] * 62], [[2.0, 3.5] + [0.0] * 62]])
    cache, scale = np.zeros((2, 1, 16, 64), np.uint8), np.zeros((2, 1), np.float32)
    O.append(x, cache, scale, [[1]], [2], [0, 2], O.E4M3)
    assert scale[1, 0] == 1 and np.array_equal(O.gather(cache, scale, [1], 2, O.E4M3)[0], x[:, 0])
    # a larger token raises the scale and moves the codes before it
    O.append(x[:1] * 4, cache, scale, [[1]], [3], [0, 1], O.E4M3)
    assert scale[1, 0] == 4 and np.array_equal(O.gather(cache, scale, [1], 3, O.E4M3)[0], np.concatenate([x[:, 0], 4 * x[0]]))


def test_attention_pins():
    """Equal keys give the mean of the visible values; one key gives its value."""
    rng = np.random.default_rng(0)
    kc = np.zeros((2, 1, 16, 64), np.uint8)
    vc = O.e4m3_codes(rng.standard_normal((2, 1, 16, 64)))
    one = np.ones((2, 1), np.float32)
    q = rng.standard_normal((3, 2, 64))
    out, lse, _, _ = O.attention(q, kc, vc, one, one, [[1, 0]], [20], [0, 3], O.E4M3, 0.125)
    v = np.concatenate([O.values(vc[1, 0], 0), O.values(vc[0, 0], 0)])
    for i, n in enumerate((18, 19, 20)):
        assert np.allclose(out[i, 0], v[:n].mean(0)) and np.allclose(lse[i], np.log(n))
    out, lse, _, _ = O.attention(q, kc, vc, one, one, [[1, 0]], [20], [0, 3], O.E4M3, 0.125, window=1)
    assert np.allclose(out[2, 1], v[19]) and np.allclose(lse, 0)
    out, lse, _, _ = O.attention(q, kc, vc, one, one, [[1, 0]], [1], [0, 3], O.E4M3, 0.125)
    assert not out[:2].any() and np.isneginf(lse[:2]).all() and np.allclose(out[2, 0], v[0])


def test_rope_pins():
    """Norms stay, opposite positions undo each other, scores go by differences."""
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal((4, 2, 16)), 100.0 ** (-np.arange(8) / 8)
    axis, pos = [0] * 5 + [1] * 3, rng.integers(0, 50, (2, 4))
    for halves in (True, False):
        y = O.rope(x, pos, f, axis, halves)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.allclose(O.rope(y, -pos, f, axis, halves), x)
        a = np.einsum("thd,thd->th", O.rope(x, pos + 7, f, axis, halves), O.rope(x[::-1], pos + 7, f, axis, halves))
        b = np.einsum("thd,thd->th", y, O.rope(x[::-1], pos, f, axis, halves))
        assert np.allclose(a, b)
