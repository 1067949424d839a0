"""Host side of the decoder-layer operators at the edges of their arguments:
bounds that are loose, lists that name no place, tensors of the wrong size.
No GPU."""
import ctypes

import pytest

import int4_group_quantized_int4g_gb300 as fl
from int4_group_quantized_int4g_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def L():
    _build.build()
    return fl.lib()


# ------------------------------------------------------------------ max_q

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (8, 4), (4, 8), (2, 16), (1, 33)])
def test_workspace_covers_every_max_q(dim, kv_heads, group):
    """The launch never reaches past what the size query answered, however
    loose the bound on a sequence's rows is."""
    for T in (1, 2, 3, 4, 5, 8, 9, 16, 31, 32, 33, 48, 64, 1000):
        for B in (1, 2, 3, 8, 48):
            size = fl.fl_kv8_attention_workspace(T, B, kv_heads * group, kv_heads, dim)
            for max_q in (1, 2, 5, 8, 9, 16, 17, 32, 33, T, T + 1, 4 * T, 128, 4096, 2 ** 29, 2 ** 31 - 1):
                rows, many, few, reach = fl.fl_kv8_test_plan(T, B, max_q, kv_heads * group, kv_heads, dim)
                assert reach <= size, (T, B, max_q)
                assert rows == min(T, max_q) * group           # no sequence has more rows than the call
                assert many == (rows > 32) and few == (rows <= 32 or B > 1)


def test_plan_refusals(L):
    out = (ctypes.c_longlong * 4)()
    assert L.fl_kv8_test_plan(4, 1, 5, 8, 1, 128, out) == 0
    for bad in ((0, 1, 5, 8, 1, 128), (4, 0, 5, 8, 1, 128), (4, 1, 0, 8, 1, 128), (4, 1, 5, 8, 3, 128), (4, 1, 5, 8, 1, 80)):
        assert L.fl_kv8_test_plan(*bad, out) == 1
    assert L.fl_kv8_test_plan(4, 1, 5, 8, 1, 128, None) == 1


def test_pages_of_a_loose_max_q():
    """A bound above the call's rows changes nothing."""
    for max_q in (3, 5, 6, 1000, 2 ** 31 - 1):
        r = fl.fl_kv8_test_pages([50, 33], [[3, 1, 4, 0], [7, 2, 5, 6]], 5, 8, 16, 0, cu_q=[0, 3, 5], max_q=max_q)
        assert (r["start"], r["rows"], r["kv"]) == (0, 3, 50) and r["write"] == (2, 2, 0) and r["read"] == (0, 4, 0)
