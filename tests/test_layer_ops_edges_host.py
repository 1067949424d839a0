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


# ---------------------------------------------------------------- lists

def test_sequences_that_name_what_is_not_there_are_left_out():
    """A length past the table, more rows than max_q, lists that fall or leave
    the call's rows: no row and no page, instead of rows at other positions."""
    table = [[3, 1], [7, 2], [0, 4]]                                  # room for 32 tokens each

    def seen(lens, cu, b, max_q=None):
        r = fl.fl_kv8_test_pages(lens, table, 9, 8, 16, b, cu_q=cu, max_q=max_q)
        return r["rows"], r["kv"], r["write"][1], r["read"][1]
    good = [20, 32, 5], [0, 3, 7, 9]
    assert [seen(*good, b) for b in range(3)] == [(3, 20, 1, 2), (4, 32, 1, 2), (2, 5, 1, 1)]
    left_out = (0, 0, 0, 0)
    for n in (33, 34, 48, 2 ** 31 - 1):
        lens = [20, n, 5]
        assert seen(lens, good[1], 1) == left_out and seen(lens, good[1], 0) == (3, 20, 1, 2) and seen(lens, good[1], 2) == (2, 5, 1, 1)
    for max_q in (1, 3):
        assert seen(*good, 1, max_q) == left_out
    assert seen(*good, 0, 3) == (3, 20, 1, 2) and seen(*good, 1, 4) == (4, 32, 1, 2)
    for cu in ([0, 3, 2, 9], [0, 3, 10, 10], [0, 3, -1, 9], [0, 3, 2 ** 31 - 1, 9], [0, 3, -2 ** 31, 9]):
        assert seen(good[0], cu, 1) == left_out and seen(good[0], cu, 0) == (3, 20, 1, 2)
    assert seen(good[0], [-1, 3, 7, 9], 0) == left_out
    assert seen([20, -5, 5], good[1], 1) == (4, 0, 0, 0)              # a negative length is no token
    assert seen([20, 99, 5], [0, 3, 3, 9], 1) == left_out             # (without rows nothing is read anyway)


def test_more_rows_a_sequence_than_max_q_is_refused(L):
    A = ctypes.c_void_p(0x10000)
    c = fl.FlKv8Cache(k=A, v=A, k_scale=A, v_scale=A, num_blocks=8, block=16, kv_heads=2, head_dim=64, format=0)
    s = fl.FlKv8Seqs(cu_q=None, kv_lens=A, block_table=A, T=8, B=2, max_q=3, max_blocks=4)
    assert L.fl_kv8_append(A, 128, A, 128, ctypes.byref(c), ctypes.byref(s), A, None) == 1
    assert L.fl_kv8_attention(A, 256, 4, ctypes.byref(c), ctypes.byref(s), 0.1, 0, A, 256, None, A, 1 << 30, None) == 1


def test_attention_refuses_an_output_over_its_queries(L):
    """q is read at any time of the call.  Rows that alternate in one buffer are
    not refused (here they fail later: there is no GPU)."""
    c = fl.FlKv8Cache(k=1 << 20, v=1 << 20, k_scale=1 << 20, v_scale=1 << 20, num_blocks=8, block=16, kv_heads=2, head_dim=64, format=0)
    base = 1 << 24

    def call(at, qs=256, os=256, T=4):   # the output starts `at` elements behind q; rows of 256
        s = fl.FlKv8Seqs(cu_q=None, kv_lens=1 << 20, block_table=1 << 20, T=T, B=1, max_q=T, max_blocks=4)
        return L.fl_kv8_attention(ctypes.c_void_p(base), qs, 4, ctypes.byref(c), ctypes.byref(s), 0.1, 0, ctypes.c_void_p(base + 2 * at), os,
                                  None, ctypes.c_void_p(1 << 20), 1 << 30, None)
    for T in (1, 4):
        for at in (0, 8, -8, 248, -248):
            assert call(at, T=T) == 1 and call(at, 512, 512, T) == 1 and call(at, 512, 256, T) == 1
    assert call(256) == 1 and call(3 * 256 + 248) == 1 and call(-3 * 256 - 248) == 1      # over another row
    assert call(512 + 8, 512, 512) == 1 and call(-512 - 8, 512, 512) == 1 and call(512 + 256 + 8, 512, 512) == 1
    assert call(1 << 20, T=1 << 15) == 1

    def free(*a, **kw):   # right as far as overlap goes
        import torch
        return torch.cuda.is_available() or call(*a, **kw) == 4
    assert free(4 * 256) and free(-4 * 256) and free(256, T=1)
    assert free(256, 512, 512) and free(-256, 512, 512) and free(512 + 256, 512, 512) and free(256, 1024, 1024)
    assert free(1 << 20, 512, 512, T=1 << 11)


def test_rmsnorm_refuses_one_place_for_both_outputs(L):
    x, a, b = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21), ctypes.c_void_p(1 << 22)

    def call(y, ro, H=256):
        return L.fl_rmsnorm(x, H, x, H, None, 1e-6, 1, 1, H, y, H, ro, H, None, None, 0, None)
    import torch
    for H in (8, 64, 256):
        assert call(a, a, H) == 1 and call(x, x, H) == 1
        assert torch.cuda.is_available() or (call(a, b, H) == 4 and call(x, b, H) == 4 and call(a, None, H) == 4)


# ---------------------------------------------------------------- binding

class Fake:
    """A tensor on a GPU, as far as the binding looks at it; nothing is launched."""

    def __init__(self, shape, dtype):
        import torch
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, torch.device("cuda", 0)

    def stride(self):
        st, n = [], 1
        for d in reversed(self.shape):
            st.insert(0, n)
            n *= d
        return tuple(st)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def calls(monkeypatch):
    """The library's calls by name, none of them made."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0
    monkeypatch.setattr(fl, "lib", lambda: Lib())
    monkeypatch.setattr(fl, "_stream", lambda stream=None: None)
    return made


def test_append_refuses_a_status_that_is_too_small(calls):
    import torch
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    args = [Fake((2, 1, 64), bf), Fake((2, 1, 64), bf), Fake((4, 1, 16, 64), u8), Fake((4, 1, 16, 64), u8), Fake((4, 1), f32),
            Fake((4, 1), f32), Fake((2, 2), i32), Fake((2,), i32)]
    for status in (Fake((1,), i32), Fake((3,), i32), Fake((15,), u8), Fake((0,), u8)):
        with pytest.raises(ValueError):
            fl.fl_kv8_append(*args, status=status)
    assert calls == []
    for status in (Fake((4,), i32), Fake((16,), u8), Fake((1 << 20,), u8)):
        fl.fl_kv8_append(*args, status=status)
    assert calls == ["fl_kv8_append"] * 3


def test_rope_refuses_positions_of_another_shape(calls):
    """Positions of three axes of dimensions, or of as many tokens in another
    order, are not read as if they were one list."""
    import torch
    q, f = Fake((6, 2, 64), torch.bfloat16), Fake((32,), torch.float64)

    def turn(shape, **kw):
        return fl.fl_rope(q, None, Fake(shape, torch.int32), f, q_out=q, **kw)
    for shape in ((1, 1, 6), (2, 3, 6), (), (5,), (6, 1), (3, 5)):
        with pytest.raises(ValueError):
            turn(shape)
    with pytest.raises(ValueError):
        turn((2, 6), sections=[10, 10, 12])
    assert calls == []
    turn((6,))
    turn((1, 6))
    turn((3, 6), sections=[10, 10, 12])
    assert calls == ["fl_rope"] * 3


def test_workspaces_under_capture_and_outgrown(monkeypatch):
    """A workspace made while a stream is captured belongs to that call alone
    (its zeros are written when the graph is replayed, not before); one that a
    larger replaces stays, for the graphs that were captured with it."""
    import gc
    import types
    import weakref

    import torch
    made, state = [], {"capturing": False}

    class Buffer:
        def __init__(self, n):
            self.n = n

        def numel(self):
            return self.n

    def zeros(n, **kw):
        b = Buffer(n)
        made.append(weakref.ref(b))
        return b
    fake = types.SimpleNamespace(zeros=zeros, uint8=torch.uint8, _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: 77),
                                 cuda=types.SimpleNamespace(is_current_stream_capturing=lambda: state["capturing"]))
    monkeypatch.setattr(fl, "_torch", lambda: fake)
    monkeypatch.setattr(fl, "_WS", {})
    monkeypatch.setattr(fl, "_OUTGROWN", [])
    dev = torch.device("cuda", 0)
    state["capturing"] = True
    a, b = fl._workspace(1000, dev), fl._workspace(1000, dev)
    assert a is not b and not fl._WS                       # each has zeros of its own in the graph
    state["capturing"] = False
    small = fl._workspace(1000, dev)
    assert small is not a and fl._workspace(900, dev) is small
    state["capturing"] = True
    assert fl._workspace(1000, dev) is small               # zero already: a captured call may use it
    large = fl._workspace(5000, dev)
    assert large is not fl._workspace(5000, dev)
    state["capturing"] = False
    ref = weakref.ref(small)
    del small
    grown = fl._workspace(1001, dev)
    gc.collect()
    assert ref() is not None and grown.numel() >= 2000     # (at least twice as large: what stays is bounded)
    assert fl._workspace(2000, dev) is grown


# ---------------------------------------------------------------- build

def test_build_checks_the_registers_of_split_kernels():
    """A compiler that gives the prompt kernel another register count fails the
    build, not the calls."""
    def log(*regs):
        return "".join(f"ptxas info    : Compiling entry function '_Z{i}k_kv8_promptILi{i}EE' for 'sm_103a'\n"
                       "ptxas info    : Function properties for x\n    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
                       f"ptxas info    : Used {r} registers, used 1 barriers\n" for i, r in enumerate(regs)) + (
            "ptxas info    : Compiling entry function '_Z9k_kv8_joinILi64EE' for 'sm_103a'\nptxas info    : Used 46 registers\n")
    _build.check_registers(log(96, 96, 96, 96), "k_kv8_prompt", 96)
    for bad in (log(96, 88), log(104), log()):
        with pytest.raises(RuntimeError, match="96 registers"):
            _build.check_registers(bad, "k_kv8_prompt", 96)
    for name, (kernel, count) in _build.REGISTERS.items():
        text = open(_build.CSRC + "/" + name).read()
        assert f"kRegs = {count}," in text and f"{kernel}(" in text
