"""The operators on feature rows on a stream of another device: tensors are checked against that stream's
device. No GPU: the operators' state stands for two devices."""
import contextlib
from types import SimpleNamespace

from topology_construction_amd import binding


def test_call_on_a_stream_of_another_device():
    ops = binding._Ops()
    now = [0]

    @contextlib.contextmanager
    def on_stream(stream):
        before, now[0] = now[0], stream.device
        yield
        now[0] = before

    ops.on_stream, ops.device, ops.stream = on_stream, lambda: now[0], lambda device: 1000 + device
    seen = []

    def f(*args):
        seen.append((now[0], args))

    ops.call(f, None, "x")
    ops.call(f, SimpleNamespace(device=1, cuda_stream=77), "x")
    ops.call(f, None, "x")
    assert seen == [(0, ("x", 0, 1000)), (1, ("x", 1, 77)), (0, ("x", 0, 1000))]
