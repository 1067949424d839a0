"""GPU parity of the decoder-layer operators at the edges of their arguments,
against the float64 oracle; tolerances as in test_gpu_layer_ops.py."""
import numpy as np
import pytest
import torch

import int4_group_quantized_int4g_gb300 as fl
from oracle import layer_oracle as O
from test_gpu_layer_ops import DEV, FMT, Cache, _bf16, _close, _cu, _i32, _np, _table

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
