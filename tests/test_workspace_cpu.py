"""The cached workspace of the Python calls (no GPU needed): CPU tensors, a
stand-in for the library whose entry points record the workspace they get."""
import contextlib
import threading

import pytest
import torch

import muon_newton_schulz_06_amd as mns
from muon_newton_schulz_06_amd import layers


class Library:
    """Sizes are fixed; `inside` runs while a call enqueues its kernels."""

    def __init__(self):
        self.need = 4096
        self.inside = lambda name, ws: None

    def size(self, *args):
        args[-1]._obj.value = self.need
        return 0

    def __getattr__(self, name):
        if name.endswith("_size"):
            return self.size

        def call(*args):
            ws = args[-3]
            self.inside(name, getattr(ws, "value", ws))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    L = Library()
    made = []  # keeps every buffer, so that no address is handed out twice
    empty = torch.empty

    def keep(*args, **kw):
        made.append(empty(*args, **kw))
        return made[-1]
    monkeypatch.setattr(mns, "load", lambda: L)
    monkeypatch.setattr(layers, "_lib", lambda: L)
    monkeypatch.setattr(layers, "_device", lambda t, name: t.device)
    monkeypatch.setattr(layers, "_on", lambda dev, stream: contextlib.nullcontext())
    for m in (mns, layers):
        monkeypatch.setattr(m, "_raw_stream", lambda index: 7)
    monkeypatch.setattr(mns, "_ws_cache", {})
    monkeypatch.setattr(torch, "empty", keep)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return L


def gated_ffn():
    w = torch.zeros((24, 16))
    mns.muon_gated_ffn(torch.zeros((4, 16)), w, w, torch.zeros((16, 24)))


def gated_ffn_grad():
    x, w = torch.zeros((4, 16)), torch.zeros((24, 16))
    mns.muon_gated_ffn_grad(x, x, w, w, torch.zeros((16, 24)), torch.zeros(64, dtype=torch.uint8))


def embedding_grad():
    mns.muon_embedding_grad(torch.zeros((4, 16)), torch.zeros(4, dtype=torch.int64), 5)


def rms_norm_grad():
    x = torch.zeros((4, 16))
    mns.muon_rms_norm_grad(x, x, torch.ones(16), torch.ones(4))


CALLS = [gated_ffn, gated_ffn_grad, embedding_grad, rms_norm_grad]


@pytest.mark.parametrize("call", CALLS)
def test_threads_on_one_stream_take_turns(fake, call):
    """Two threads on one stream: while one enqueues a call's kernels, the
    other enqueues none that use the same buffer (they would come between)."""
    both = threading.Barrier(2)
    meet = threading.Barrier(2)
    lock, busy, shared = threading.Lock(), {}, []

    def inside(name, ws):
        with lock:
            busy[ws] = busy.get(ws, 0) + 1
            shared.append(busy[ws])
        try:  # the other thread has this long to get into its call, too
            meet.wait(0.5)
        except threading.BrokenBarrierError:
            pass
        with lock:
            busy[ws] -= 1
    fake.inside = inside

    def run():
        both.wait()
        call()
    ts = [threading.Thread(target=run) for _ in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert shared == [1, 1]


def test_buffer_is_reused_and_grows(fake):
    """One buffer per stream, kept from call to call, replaced by a larger
    one when a call needs it, dropped on request."""
    seen = []
    fake.inside = lambda name, ws: seen.append(ws)
    gated_ffn()
    embedding_grad()
    assert seen[0] == seen[1]
    fake.need = 8192
    gated_ffn()
    fake.need = 4096
    gated_ffn()
    assert seen[2] != seen[0] and seen[3] == seen[2]
    mns.release_workspace()
    gated_ffn()
    assert seen[4] != seen[3]


def test_failing_call_lets_the_next_one_in(fake):
    """A call that raises inside holds nothing up."""
    def inside(name, ws):
        raise RuntimeError("inside")
    fake.inside = inside
    with pytest.raises(RuntimeError, match="inside"):
        gated_ffn()
    fake.inside = lambda name, ws: None
    t = threading.Thread(target=gated_ffn, daemon=True)
    t.start()
    t.join(10)
    assert not t.is_alive()


@pytest.mark.parametrize("call", CALLS)
def test_not_cached_while_capturing(fake, monkeypatch, call):
    """A call that is captured into a graph takes a buffer of its own from
    the capture's memory: neither one that eager calls use, and may replace by
    a larger one, nor one that another captured call has."""
    seen = []
    fake.inside = lambda name, ws: seen.append(ws)
    call()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    call()
    call()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    call()
    assert seen[3] == seen[0] and len(set(seen[:3])) == 3


def test_captured_call_on_a_given_stream(fake, monkeypatch):
    """Whether to capture is a matter of the stream the call runs on."""
    on = []

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()
    side = type("Stream", (), {"cuda_stream": 9})()
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: on == [side])
    dev = torch.device("cpu")
    with mns._workspace(4096, dev, None, side) as (buf, n):
        assert n == 4096
    with mns._workspace(4096, dev, None) as (other, _):
        assert other is not buf
    with mns._workspace(4096, dev, None, side) as (again, _):
        assert again is not buf and again is not other
    with mns._workspace(4096, dev, None) as (last, _):
        assert last is other
