"""Calls on a stream of their own that leave out their outputs and workspace, while the caller's
stream is busy and hands out freed memory: the same results, and nobody else's memory touched."""
import pytest
import torch

from block_sparse_attention_oam_b200 import stem as S
from block_sparse_attention_oam_b200 import workloads as W
from tests import stem_testlib as T
from tests import test_gpu_decode as D
from tests import test_gpu_evict as E

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def _beside(call, sizes):
    """Runs call(stream) ten times, each behind 1 ms of work on the caller's stream that the call
    does not wait for, and takes memory of `sizes` bytes on the caller's stream after each.
    Returns what the calls returned; fails where that memory was written."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, held = [], []
    for _ in range(10):
        torch.cuda._sleep(2_000_000)
        got.append(call(side))
        held.append([torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes])
    torch.cuda.synchronize()
    assert all((t == 0xA5).all() for ts in held for t in ts)
    return got


@pytest.mark.parametrize("kw", [dict(lens=[9000, 40], weights=True), dict(lens=[30, 700] * 20, prefix=2000)])
def test_decode(kw):
    s = D.Setup(Hq=8, Hkv=2, d=128, seed=50, **kw)
    want = s.call().clone()
    rows = len(s.lens) * s.Hq * s.d * 2
    got = _beside(lambda side: S.stem_decode(s.dec, s.q, s.cache, s.kv_lens, prefix_table=s.prefix_table, weights_in=s.w_in,
                                             weights_out=s.w_out, stream=side), [s.dec.workspace_bytes(), rows])
    assert all(torch.equal(x, want) for x in got)


def test_evict():
    s = E.Setup([9000, 700], Hkv=2, d=128, budget=300, sink=4, recent=50, seed=51)
    want, lens = S.stem_evict(s.ev, s.src, s.kv_lens, s.w, s.dst)
    got = _beside(lambda side: S.stem_evict(s.ev, s.src, s.kv_lens, s.w, s.dst, stream=side),
                  [s.ev.workspace_bytes(), want.numel() * 4, 8])
    assert all(torch.equal(k, want) and torch.equal(n, lens) for k, n in got)


def test_prefill():
    wl = W.QWEN_32K.with_(name="side_stream", seqlens=(2048, 700), num_q_heads=8, num_kv_heads=2, seed=52)
    inp = W.make_inputs(wl)
    prob, dev = S.problem_for(wl, inp), T.to_device(inp)
    want = S.stem_attention(prob, dev["q"], dev["k"], dev["v"])
    rp, ci = S.stem_score_select(prob, dev["q"], dev["k"], dev["v"])
    sizes = [prob.sizes()["workspace_bytes"], want.numel() * 2]
    got = _beside(lambda side: S.stem_attention(prob, dev["q"], dev["k"], dev["v"], stream=side), sizes)
    assert all(torch.equal(x, want) for x in got)
    got = _beside(lambda side: S.stem_score_select(prob, dev["q"], dev["k"], dev["v"], stream=side), sizes + [rp.numel() * 4, ci.numel() * 4])
    assert all(torch.equal(a, rp) and torch.equal(b, ci) for a, b in got)


def test_a_captured_path_leaves_other_memory_alone():
    """A captured path that made its own workspace: what is allocated afterwards is not its to write."""
    wl = W.QWEN_32K.with_(name="captured_alone", seqlens=(2048, 700), num_q_heads=8, num_kv_heads=2, seed=53)
    inp = W.make_inputs(wl)
    prob, dev = S.problem_for(wl, inp), T.to_device(inp)
    want = S.stem_attention(prob, dev["q"], dev["k"], dev["v"])
    graph, out = S.capture_attention(prob, dev["q"], dev["k"], dev["v"])
    n = prob.sizes()["workspace_bytes"]
    held = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert all((t == 0xA5).all() for t in held)
