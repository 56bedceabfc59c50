"""Where the calls take the memory of the outputs and workspaces that they make
when a stream is passed: from that stream's own pool, whatever the current
stream is.  Runs without a GPU, on stand-ins for torch's streams and allocator."""
import ast
import contextlib

import pytest
import torch

from conftest import build_lib

CURRENT, PASSED = 0x7000, 0x9000


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = int(handle)


class Made:
    def __init__(self, on, n):
        self.on, self.n, self.recorded = on, n, []

    def numel(self):
        return self.n

    def record_stream(self, s):
        self.recorded.append(s.cuda_stream)


@pytest.fixture
def w(monkeypatch):
    build_lib()
    import weight_transfer_gb300 as m
    now = [Stream(CURRENT)]

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch, "empty", lambda shape, **kw: Made(now[-1].cuda_stream, int(torch.Size(
        shape if isinstance(shape, (tuple, list)) else (shape,)).numel())))
    return m


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_memory_of_the_passed_stream(w, how):
    s = Stream(PASSED) if how == "stream" else PASSED
    t = w._new((4, 5), torch.uint8, torch.device("cuda"), s)
    assert t.on == PASSED and t.recorded == [CURRENT]
    t = w._new(64, torch.uint8, torch.device("cuda"), s, kept=False)
    assert t.on == PASSED and t.recorded == []
    assert w._new((0, 8), torch.uint8, torch.device("cuda"), s).recorded == []


@pytest.mark.parametrize("s", [None, CURRENT, Stream(CURRENT)])
def test_memory_of_the_current_stream(w, s):
    t = w._new((4, 5), torch.uint8, torch.device("cuda"), s)
    assert t.on == CURRENT and t.recorded == []


@pytest.mark.parametrize("s", [0, 1])
def test_legacy_default_stream(w, s):
    """Handles 0 and 1 both name the legacy default stream, whose memory is that of torch's default stream."""
    assert w._new((4, 5), torch.uint8, torch.device("cuda"), s).on == 0


def test_every_call_takes_its_memory_there():
    """No function of the binding that takes a stream asks torch for memory by itself."""
    build_lib()
    import weight_transfer_gb300 as m
    with open(m.__file__) as f:
        tree = ast.parse(f.read())
    bad = []
    for fn in tree.body:
        if isinstance(fn, ast.FunctionDef) and fn.name not in ("_new", "_out") and "stream" in [a.arg for a in fn.args.args]:
            bad += [f"{fn.name}: {ast.unparse(c)}" for c in ast.walk(fn) if isinstance(c, ast.Call)
                    and isinstance(c.func, ast.Attribute) and isinstance(c.func.value, ast.Name) and c.func.value.id == "torch"]
    assert not bad, bad
