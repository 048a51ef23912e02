"""Where a call with a stream of its own allocates what its caller left out, seen without a GPU:
the allocator, the streams and the library are stand-ins that write down what happens."""
import contextlib
import gc
import weakref

import pytest
import torch

from block_sparse_attention_oam_b200 import stem as S

DEV = torch.device("cuda", 0)


class Stream:
    def __init__(self, name, device=DEV):
        self.name, self.device, self.cuda_stream = name, device, 64


class Tensor:
    """Device memory: where it was allocated, and which streams it was recorded on."""
    is_cuda = True

    def __init__(self, shape, log, device=DEV, how="given"):
        self.shape, self.device, self.how = shape, device, how
        self.home, self.recorded = log.current, []

    def record_stream(self, stream):
        self.recorded.append(stream)

    def numel(self):
        return 1 << 20

    def data_ptr(self):
        return 256

    def is_contiguous(self):
        return True


class Log:
    def __init__(self, monkeypatch):
        self.mine = self.current = Stream("the caller's")
        self.made, self.calls = [], []

        @contextlib.contextmanager
        def on(stream):
            was, self.current = self.current, stream
            yield
            self.current = was

        def make(how):
            def f(shape, dtype=None, device=None):
                assert torch.device(device).type == "cuda"
                self.made.append(Tensor(shape, self, how=how))
                return self.made[-1]
            return f

        def entry(*args):
            self.calls.append(args)
            return 0

        class Lib:
            def __getattr__(_, name):
                if name.endswith("workspace_size"):
                    return lambda *a: 4096
                return entry

        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch, "empty", make("empty"))
        monkeypatch.setattr(torch, "zeros", make("zeros"))
        monkeypatch.setattr(S, "_native", (entry, 0, entry, 0))
        monkeypatch.setattr(S, "_lib", Lib())
        self.t = Tensor((4, 2, 64), self)
        self.kv = S.PagedKV(*(Tensor(s, self) for s in ((9, 64, 2, 64), (9, 64, 2, 64), (4, 16))))


@pytest.fixture
def log(monkeypatch):
    return Log(monkeypatch)


def _problem(monkeypatch):
    prob = S.Problem([0, 4], 2, 2, 64, 64)
    monkeypatch.setattr(S.Problem, "sizes", lambda self: dict(num_rows=2, scores_per_head=3, nnz_per_head=2, total_tokens=4,
                                                              workspace_bytes=4096, list_heads=2))
    return prob


def calls(log, monkeypatch):
    """Every entry that takes a stream, with nothing but its inputs."""
    p, t, kv = _problem(monkeypatch), log.t, log.kv
    return {
        "stem_decode": lambda s: S.stem_decode(S.Decode(4, 2, 2, 64, max_kv_len=1000), t, kv, t, stream=s),
        "stem_evict": lambda s: S.stem_evict(S.Evict(4, 2, 64, max_kv_len=1000, budget=64), kv, t, t, kv, stream=s),
        "stem_score": lambda s: S.stem_score(p, t, t, t, stream=s),
        "stem_select": lambda s: S.stem_select(p, t, stream=s),
        "stem_score_select": lambda s: S.stem_score_select(p, t, t, t, stream=s),
        "bsa_prefill": lambda s: S.bsa_prefill(p, t, t, t, t, t, stream=s),
        "bsa_dense_prefill": lambda s: S.bsa_dense_prefill(p, t, t, t, stream=s),
        "stem_attention": lambda s: S.stem_attention(p, t, t, t, stream=s),
        "stem_attention_noalloc": lambda s: S.stem_attention_noalloc(p, t, t, t, stream=s),
    }


NAMES = ["stem_decode", "stem_evict", "stem_score", "stem_select", "stem_score_select", "bsa_prefill", "bsa_dense_prefill",
         "stem_attention", "stem_attention_noalloc"]


@pytest.mark.parametrize("name", NAMES)
def test_what_is_left_out_is_allocated_on_the_calls_stream(log, monkeypatch, name):
    """The workspace is zeroed in the order of the kernels' stream and goes back to that stream's
    pool; outputs are the caller's to read on its own stream."""
    side = Stream("the call's")
    got = calls(log, monkeypatch)[name](side)
    assert log.calls and log.made
    assert all(t.home is side for t in log.made)
    for t in got if isinstance(got, tuple) else (got,):
        assert t in log.made and t.recorded == [log.mine]
    assert log.current is log.mine


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_everything_is_on_the_current_one(log, monkeypatch, name):
    calls(log, monkeypatch)[name](None)
    assert log.calls and log.made
    assert all(t.home is log.mine and not t.recorded for t in log.made)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(log, monkeypatch, name):
    with pytest.raises(ValueError, match="cuda:1"):
        calls(log, monkeypatch)[name](Stream("elsewhere", torch.device("cuda", 1)))
    assert not log.calls


def test_a_captured_path_keeps_its_workspace(log, monkeypatch):
    """Replays write the workspace, so it lives as long as the graph, given or not."""
    @contextlib.contextmanager
    def on(stream):
        yield

    class Graph:
        pass

    side = Stream("the first call's")
    side.wait_stream = lambda s: None
    log.mine.wait_stream = lambda s: None
    monkeypatch.setattr(torch.cuda, "Stream", lambda device=None: side)
    monkeypatch.setattr(torch.cuda, "CUDAGraph", Graph)
    monkeypatch.setattr(torch.cuda, "graph", on)
    graph, _ = S.capture_attention(_problem(monkeypatch), log.t, log.t, log.t)
    ws, = [weakref.ref(t) for t in log.made if t.how == "zeros"]
    log.made.clear()
    log.calls.clear()
    gc.collect()
    assert ws() is not None
    del graph
    gc.collect()
    assert ws() is None
