"""Host threads that share a stream share its workspace, in which a call's
launches hand partial sums to one another: their calls take turns."""

import threading
import time
from types import SimpleNamespace

import quantized_base_rank_amd as qb


def _in_threads(n, fn):
    errors = []

    def body(i):
        try:
            fn(i)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    ts = [threading.Thread(target=body, args=(i,)) for i in range(n)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


def test_calls_on_one_stream_take_turns(monkeypatch):
    shared = object()
    monkeypatch.setattr(qb, "_capturing", lambda: False)
    monkeypatch.setattr(qb, "_WS_STREAM", {(0, 5): shared})
    inside, most = [], []

    def call(ws):
        assert ws is shared
        inside.append(1)
        most.append(len(inside))
        time.sleep(0.005)  # (a foreign call: other threads run meanwhile)
        inside.pop()
        return 0

    dev = SimpleNamespace(index=0)
    _in_threads(6, lambda i: [qb._call_with_workspace(call, lambda: 1, dev, 5, None) for _ in range(3)])
    assert max(most) == 1


def test_a_workspace_that_grows_is_not_swapped_under_another_call(monkeypatch):
    """The first thread's call runs on the small workspace while the second's asks for a larger one."""
    order = []
    monkeypatch.setattr(qb, "_capturing", lambda: False)
    monkeypatch.setattr(qb, "_WS_STREAM", {(0, 5): "small"})

    def grown(device, stream, nbytes):
        order.append("grown")
        qb._WS_STREAM[(0, 5)] = "large"
        return "large"
    monkeypatch.setattr(qb, "_stream_workspace", grown)
    started = threading.Event()

    def first(ws):
        assert ws == "small"
        started.set()
        time.sleep(0.02)
        order.append("first done")
        return 0

    def second(ws):
        return 0 if ws == "large" else qb.QLIN_E_WORKSPACE

    dev = SimpleNamespace(index=0)

    def run(i):
        if i == 0:
            qb._call_with_workspace(first, lambda: 1, dev, 5, None)
        else:
            assert started.wait(5)
            qb._call_with_workspace(second, lambda: 1, dev, 5, None)
    _in_threads(2, run)
    assert order == ["first done", "grown"]


def test_calls_on_different_streams_do_not_wait(monkeypatch):
    monkeypatch.setattr(qb, "_capturing", lambda: False)
    monkeypatch.setattr(qb, "_WS_STREAM", {(0, 5): "a", (0, 6): "b", (1, 5): "c"})
    together = threading.Barrier(3, timeout=5)  # broken unless all three are inside at once

    def call(ws):
        together.wait()
        return 0
    keys = [(0, 5), (0, 6), (1, 5)]
    _in_threads(3, lambda i: qb._call_with_workspace(call, lambda: 1, SimpleNamespace(index=keys[i][0]), keys[i][1], None))


class _Tensor:
    """What the binding asks of a device tensor, without a device."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def numel(self):
        return 1 << 20


def test_layer_calls_on_the_device_s_workspace_take_turns(monkeypatch):
    import torch
    inside, most = [], []

    def native(*args):
        inside.append(1)
        most.append(len(inside))
        time.sleep(0.005)
        inside.pop()
        return 0
    fake = SimpleNamespace(qlin_fwd=native, qlin_bwd=native, qlin_workspace_bytes=lambda *a: 1)
    monkeypatch.setattr(qb, "lib", lambda: fake)
    monkeypatch.setattr(qb, "_stream", lambda device: 0)
    monkeypatch.setattr(qb, "workspace", lambda device, nbytes: _Tensor(torch.uint8, 1 << 20))
    bf = torch.bfloat16
    dev = torch.device("cuda", 0)
    x, A, B, dy = _Tensor(bf, 4, 64), _Tensor(bf, 2, 64), _Tensor(bf, 16, 2), _Tensor(bf, 4, 16)
    u = _Tensor(torch.float32, 4, 2)
    for t in (x, A, B, dy, u):
        t.device = dev
    w = qb.QWeight(qb.QLIN_FMT_NF4, 64, 0, 16, 64, _Tensor(torch.uint8, 16, 32), absmax=_Tensor(torch.float32, 16))

    def body(i):
        for _ in range(3):
            if i % 2 == 0:
                qb.qlin_fwd(w, x, A, B, 2, 1.0, y=dy, u_out=u)
            else:
                qb.qlin_bwd(w, x, A, B, 2, 1.0, dy, u_saved=u, dx=x, dA=A, dB=B)
    _in_threads(6, body)
    assert max(most) == 1 and len(most) == 18
