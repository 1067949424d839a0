"""Host side of the serving operators at the edges of their use: several threads,
tensors of other devices, outputs over inputs, pools that are full.  No GPU."""
import threading
import types

import torch

import int4_group_quantized_int4g_gb300 as fl


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
