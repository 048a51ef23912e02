"""stem_evict on the GPU: the kept positions, weights and lengths exactly those of the
oracle's rule, the K/V rows moved bit for bit, and nothing else written; then a run as a
serving loop makes it (prefill, decoding that collects weights, eviction, decoding on)."""
import numpy as np
import pytest
import torch

from block_sparse_attention_oam_b200 import stem as S
from block_sparse_attention_oam_b200 import workloads as W
from oracle import stem_oracle as O
from tests.test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

PAGE = S.PAGE_SIZE


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def _bytes(t):
    return t.view(torch.uint8)


class Setup:
    def __init__(self, lens, Hkv, d, budget, sink=0, recent=0, dtype="bf16", kind="tail", max_kv_len=None, seed=0,
                 one_cache=False):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.d, self.budget, self.sink, self.recent = list(lens), Hkv, d, budget, sink, recent
        B = len(self.lens)
        cap = max(self.lens + [1]) if max_kv_len is None else max_kv_len
        pages, fresh = -(-cap // PAGE), -(-min(budget, cap) // PAGE)
        tt = torch.float8_e4m3fn if dtype == "fp8_e4m3" else torch.bfloat16
        es = 1 if dtype == "fp8_e4m3" else 2
        slots = B * pages + (B * fresh if one_cache else 0) + 2
        perm = rng.permutation(slots).astype(np.int32)

        def noise(n):   # any bytes: rows are moved, not read
            g = torch.Generator("cuda").manual_seed(seed)
            return torch.randint(0, 256, (n, PAGE, Hkv, d * es), dtype=torch.uint8, device="cuda", generator=g).view(tt)

        k, v = noise(slots), noise(slots)
        _bytes(v).bitwise_xor_(0x5A)
        self.src = S.PagedKV(k, v, torch.from_numpy(perm[: B * pages].reshape(B, pages).copy()).cuda())
        if one_cache:
            t = perm[B * pages: B * pages + B * fresh].reshape(B, fresh).copy()
            self.dst = S.PagedKV(k, v, torch.from_numpy(t).cuda())
        else:
            t = rng.permutation(B * fresh + 1).astype(np.int32)[: B * fresh].reshape(B, fresh).copy()
            self.dst = S.PagedKV(noise(B * fresh + 1), noise(B * fresh + 1), torch.from_numpy(t).cuda())
        shape = (B, Hkv, cap + 1)
        w = rng.random(shape).astype(np.float32) ** 8
        if kind == "ties":
            w = rng.integers(0, 3, shape).astype(np.float32)
        elif kind == "equal":
            w[:] = 0.25
        elif kind == "odd":     # NaN, infinities, zeros of both signs, negatives, subnormals
            w = rng.choice(np.array([np.nan, -np.inf, np.inf, 0.0, -0.0, -1.0, 1.0, 1e-40, 2e-40], dtype=np.float32), shape)
        elif kind == "close":   # differ in the last bits only
            w = (np.float32(1.0) + rng.integers(0, 700, shape).astype(np.float32) * np.float32(2.0 ** -23)).astype(np.float32)
        self.w = torch.from_numpy(w).cuda()
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.ev = S.Evict(B, Hkv, d, max_kv_len=cap, budget=budget, sink=sink, recent=recent, dtype=dtype)

    def check(self):
        B, Hkv, budget = len(self.lens), self.Hkv, self.budget
        src_k, src_v = _bytes(self.src.k_cache).cpu(), _bytes(self.src.v_cache).cpu()
        want_k, want_v = _bytes(self.dst.k_cache).cpu(), _bytes(self.dst.v_cache).cpu()
        st, dt, w = self.src.block_table.cpu().numpy(), self.dst.block_table.cpu().numpy(), self.w.cpu().numpy()
        want_keep = np.full((B, Hkv, budget), -1, dtype=np.int32)
        w_out = torch.full((B, Hkv, budget + 2), -5.0, device="cuda")
        want_w = w_out.cpu().numpy()
        for b, n in enumerate(self.lens):
            for h in range(Hkv):
                kept = O.evict_keep(w[b, h], n, budget, self.sink, self.recent)
                m = len(kept)
                want_keep[b, h, :m] = kept
                want_w[b, h, :m] = w[b, h, kept]
                to, frm = np.arange(m), kept
                want_k[dt[b, to // PAGE], to % PAGE, h] = src_k[st[b, frm // PAGE], frm % PAGE, h]
                want_v[dt[b, to // PAGE], to % PAGE, h] = src_v[st[b, frm // PAGE], frm % PAGE, h]
        keep = torch.full((B, Hkv, budget), 77, dtype=torch.int32, device="cuda")
        ws = S.evict_workspace(self.ev)
        got, lens = S.stem_evict(self.ev, self.src, self.kv_lens, self.w, self.dst, weights_out=w_out, keep=keep, ws=ws)
        assert S.query_status(ws) == S.STEM_OK
        assert np.array_equal(got.cpu().numpy(), want_keep)
        assert lens.cpu().tolist() == [min(n, budget) for n in self.lens]
        assert np.array_equal(w_out.cpu().numpy().view(np.int32), want_w.view(np.int32))
        assert torch.equal(_bytes(self.dst.k_cache).cpu(), want_k) and torch.equal(_bytes(self.dst.v_cache).cpu(), want_v)


CASES = {
    "one_of_two": dict(lens=[2], Hkv=1, d=64, budget=1),
    "nothing_cached": dict(lens=[0, 0], Hkv=2, d=128, budget=5),
    "all_fit": dict(lens=[64, 1, 100, 0], Hkv=2, d=128, budget=100),
    "one_over": dict(lens=[101, 100, 99], Hkv=3, d=64, budget=100, sink=1, recent=1),
    "odd": dict(lens=[700, 65, 63, 1], Hkv=2, d=128, budget=63, sink=4, recent=10),
    "only_ends": dict(lens=[700, 30], Hkv=2, d=64, budget=20, sink=5, recent=15),
    "only_recent": dict(lens=[700], Hkv=1, d=128, budget=20, recent=20),
    "only_sink": dict(lens=[700], Hkv=1, d=128, budget=20, sink=20),
    "ties": dict(lens=[5000, 900], Hkv=2, d=64, budget=400, sink=3, recent=7, kind="ties"),
    "equal": dict(lens=[5000, 513], Hkv=2, d=64, budget=512, kind="equal"),
    "special_values": dict(lens=[3000, 700, 90], Hkv=4, d=64, budget=80, sink=2, recent=3, kind="odd"),
    "special_values_most": dict(lens=[3000, 700, 90], Hkv=4, d=64, budget=650, kind="odd"),
    "close": dict(lens=[20000], Hkv=2, d=64, budget=5001, sink=4, recent=64, kind="close"),
    "long_one_unit": dict(lens=[40001], Hkv=1, d=64, budget=9000, sink=4, recent=64),
    "long_gqa": dict(lens=[17000, 300, 9000], Hkv=8, d=128, budget=4097, sink=64, recent=500),
    "many": dict(lens=list(range(0, 400, 2)), Hkv=1, d=64, budget=120, sink=4, recent=30),
    "fp8": dict(lens=[700, 64, 5000], Hkv=8, d=128, budget=130, sink=4, recent=32, dtype="fp8_e4m3"),
    "one_cache": dict(lens=[700, 130, 64], Hkv=2, d=128, budget=100, sink=4, recent=30, one_cache=True),
    "bound_above_lengths": dict(lens=[300, 20], Hkv=2, d=64, budget=100, max_kv_len=30000),
    "budget_above_bound": dict(lens=[300, 20], Hkv=2, d=64, budget=5000),
    "longest": dict(lens=[262144, 70], Hkv=1, d=64, budget=30000, sink=4, recent=100),
    "longest_equal": dict(lens=[262144], Hkv=1, d=64, budget=200000, kind="equal"),
    "over_128k": dict(lens=[140001], Hkv=2, d=64, budget=1000, sink=4, recent=100, kind="odd"),
    "most_sequences": dict(lens=[b % 200 for b in range(1024)], Hkv=1, d=64, budget=90, recent=9),
    "many_heads": dict(lens=[200, 90], Hkv=200, d=64, budget=70, recent=8),
}


@pytest.mark.parametrize("name", list(CASES))
def test_evict_matches_oracle(name):
    Setup(seed=sum(map(ord, name)), **CASES[name]).check()


def test_captured_eviction_follows_the_lengths():
    s = Setup([9000, 700], Hkv=2, d=128, budget=300, sink=4, recent=50, seed=3)
    ws = S.evict_workspace(s.ev)
    keep, lens = S.stem_evict(s.ev, s.src, s.kv_lens, s.w, s.dst, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.stem_evict(s.ev, s.src, s.kv_lens, s.w, s.dst, kv_lens_out=lens, keep=keep, ws=ws)
    for new in ([9000, 700], [301, 0], [100, 5000]):
        s.kv_lens.copy_(torch.tensor(new, dtype=torch.int32))
        _bytes(s.dst.k_cache).zero_()
        g.replay()
        a, l, k = keep.clone(), lens.clone(), s.dst.k_cache.clone()
        _bytes(s.dst.k_cache).zero_()
        want, want_l = S.stem_evict(s.ev, s.src, s.kv_lens, s.w, s.dst, ws=ws)
        assert torch.equal(a, want) and torch.equal(l, want_l) and torch.equal(_bytes(k), _bytes(s.dst.k_cache))
        assert l.tolist() == [min(n, 300) for n in new]


def test_writes_only_its_buffers():
    s = Setup([700, 64, 5000, 0], Hkv=2, d=128, budget=130, sink=4, recent=32, seed=4)
    shape = tuple(s.dst.k_cache.shape)
    gk, gv = Guarded(shape, torch.bfloat16), Guarded(shape, torch.bfloat16)
    gt, gl = Guarded((4, 2, 130), torch.int32), Guarded((4,), torch.int32)
    gw = Guarded((4, 2, 130), torch.float32)
    ws = Guarded((s.ev.workspace_bytes(),), torch.uint8)
    ws.t.zero_()
    before = [t.clone() for t in (_bytes(s.src.k_cache), _bytes(s.src.v_cache), s.w, s.kv_lens)]
    S.stem_evict(s.ev, s.src, s.kv_lens, s.w, S.PagedKV(gk.t, gv.t, s.dst.block_table), kv_lens_out=gl.t,
                 weights_out=gw.t, keep=gt.t, ws=ws.t)
    assert S.query_status(ws.t) == S.STEM_OK
    assert all(g.intact() for g in (gk, gv, gt, gl, gw, ws))
    for x, y in zip(before, (_bytes(s.src.k_cache), _bytes(s.src.v_cache), s.w, s.kv_lens)):
        assert torch.equal(x, y)


def test_bad_pages_and_lengths_are_reported():
    """A source page outside its cache is read as slot 0, a destination page outside is not
    written; the sequence beside them is right."""
    s = Setup([130, 100], Hkv=2, d=64, budget=70, seed=5)
    S.stem_evict(s.ev, s.src, s.kv_lens, s.w, s.dst)
    good = _bytes(s.dst.k_cache)[s.dst.block_table[1].long()].clone()

    def bad_call(src=s.src, dst=s.dst, lens=s.kv_lens):
        _bytes(s.dst.k_cache).fill_(9)
        ws = S.evict_workspace(s.ev)
        _, n = S.stem_evict(s.ev, src, lens, s.w, dst, ws=ws)
        with pytest.raises(S.StemError) as e:
            S.query_status(ws)
        assert e.value.status == S.STEM_ERR_BOUNDS
        k = _bytes(s.dst.k_cache)
        got = k[s.dst.block_table[1].long()].flatten(0, 1)[:70]
        assert torch.equal(got, good.flatten(0, 1)[:70])
        return k, n

    for bad in (-1, s.src.k_cache.shape[0]):
        t = s.src.block_table.clone()
        t[0, :2] = bad
        bad_call(src=S.PagedKV(s.src.k_cache, s.src.v_cache, t))
    for bad in (-1, s.dst.k_cache.shape[0]):
        t = s.dst.block_table.clone()
        t[0, 0] = bad
        k, _ = bad_call(dst=S.PagedKV(s.dst.k_cache, s.dst.v_cache, t))
        assert (k[s.dst.block_table[0, 0].long()] == 9).all()
    for bad in (-3, 131):
        lens = s.kv_lens.clone()
        lens[0] = bad
        _, n = bad_call(lens=lens)
        assert n.tolist() == [max(0, min(70, bad)), 70]


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_serving_loop(dtype):
    """Prefill over a paged cache, three decoding steps that collect weights, eviction to
    fresh pages of the same cache, one more step on what is left: every step against the
    oracle on the rows that the loop's bookkeeping says are cached."""
    fp8 = dtype == "fp8_e4m3"
    wl = (W.LONG_128K_FP8 if fp8 else W.PAGED_VARLEN).with_(
        name="loop", seqlens=(1024, 300), num_q_heads=8, num_kv_heads=2, paged=True, seed=41)
    inp = W.make_inputs(wl)
    prob = S.problem_for(wl, inp)
    spare = 2 * 2 + 2 * 3
    tt = inp.k_cache.dtype
    grow = lambda c: torch.cat([_bytes(c), torch.zeros((spare,) + tuple(_bytes(c).shape[1:]), dtype=torch.uint8)]).view(tt).cuda()  # noqa: E731
    kc, vc = grow(inp.k_cache), grow(inp.v_cache)
    slots = inp.k_cache.shape[0]
    table = np.zeros((2, 18), dtype=np.int32)
    table[:, :16] = np.maximum(inp.block_table, 0)
    table[0, 16:18] = [slots, slots + 1]
    table[1, 5:7] = [slots + 2, slots + 3]
    cache = S.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    q = inp.q.cuda()
    ws = S.workspace(prob)
    S.stem_attention(prob, q, q, q, paged=cache_for_prefill(cache, inp), ws=ws)
    assert S.query_status(ws) == S.STEM_OK

    scales = dict(q_scale=inp.q_scale, k_scale=inp.k_scale, v_scale=inp.v_scale) if fp8 else {}
    kv = [[inp.dequant(x)[t0:t1] for x in ("k", "v")] for t0, t1 in ((0, 1024), (1024, 1324))]
    kv = [[np.stack([x[:, h] for h in range(2)]) for x in pair] for pair in kv]      # [Hkv, n, d]
    rng = np.random.default_rng(1)

    def codes(x, name):
        t = torch.from_numpy(x.astype(np.float32))
        t = (t / scales[name]).clamp(-448, 448).to(tt) if fp8 else t.to(tt)   # codes saturate
        return t, t.float().numpy().astype(np.float64) * scales.get(name, 1.0)

    lens = torch.tensor([1024, 300], dtype=torch.int32, device="cuda")
    cap = 18 * PAGE
    acc = torch.zeros((2, 2, cap), device="cuda")
    want_acc = [np.zeros((2, 1024 + 3)), np.zeros((2, 300 + 3))]
    dec = S.Decode(2, 8, 2, 128, max_kv_len=cap, dtype=dtype, weights=True, **scales)
    dws = S.decode_workspace(dec)

    def step(cache, lens, dec, dws, acc):
        at = lens.tolist()
        qc, qv = codes(rng.standard_normal((2, 8, 128)) * 0.3, "q_scale")
        for b in range(2):
            nk, nkv = codes(rng.standard_normal((2, 128)) * 0.3, "k_scale")
            nv, nvv = codes(rng.standard_normal((2, 128)), "v_scale")
            slot = int(cache.block_table[b, at[b] // PAGE])
            _bytes(cache.k_cache)[slot, at[b] % PAGE] = _bytes(nk).cuda()
            _bytes(cache.v_cache)[slot, at[b] % PAGE] = _bytes(nv).cuda()
            kv[b] = [np.concatenate([kv[b][0], nkv[:, None]], 1), np.concatenate([kv[b][1], nvv[:, None]], 1)]
        lens += 1
        lse = torch.empty((8, 2), device="cuda")
        out = S.stem_decode(dec, qc.cuda(), cache, lens, weights_in=acc, weights_out=acc, lse=lse, ws=dws)
        assert S.query_status(dws) == S.STEM_OK
        for b in range(2):
            k, v = (x.transpose(1, 0, 2) for x in kv[b])
            ref, ref_lse, w, mean_abs, size = O.decode_rows(qv[b:b + 1], k, v, 128 ** -0.5)
            # bounds as derived beside the decode tests' check()
            e = 128 * 2.0 ** -22 * size.max() + 2.0 ** -18 * (1 + np.abs(ref_lse).max())
            u = 2.0 ** -11 + len(k) * 2.0 ** -25 * np.abs(v).max() / mean_abs.min() if fp8 else 2.0 ** -8
            lim = 2.0 ** -8 * np.abs(ref) + (u + 2 * e + len(k) * 2.0 ** -22) * mean_abs * 1.01
            assert (np.abs(out[b].float().cpu().numpy() - ref[0]) <= lim[0]).all()
            yield b, w, e

    for i in range(3):
        for b, w, e in step(cache, lens, dec, dws, acc):
            want_acc[b][:, : w.shape[1]] += w
            got = acc[b, :, : w.shape[1]].cpu().numpy()
            assert (np.abs(got - want_acc[b][:, : w.shape[1]]) <= 4 * (e + 2.0 ** -22) * (want_acc[b][:, : w.shape[1]] + 1e-30)).all()
    budget = 160
    fresh = torch.tensor([[slots + 4, slots + 6, slots + 8], [slots + 5, slots + 7, slots + 9]], dtype=torch.int32, device="cuda")
    ev = S.Evict(2, 2, 128, max_kv_len=cap, budget=budget, sink=4, recent=32, dtype=dtype)
    small = S.PagedKV(kc, vc, fresh)
    acc2 = torch.zeros((2, 2, 3 * PAGE), device="cuda")
    before = acc.clone()
    keep, lens2 = S.stem_evict(ev, cache, lens, acc, small, weights_out=acc2)
    keep = keep.cpu().numpy()
    for b, n in enumerate(lens.tolist()):
        for h in range(2):
            assert np.array_equal(keep[b, h], O.evict_keep(before[b, h].cpu().numpy(), n, budget, 4, 32))
        kv[b] = [np.stack([x[h][keep[b, h]] for h in range(2)]) for x in kv[b]]
    dec2 = S.Decode(2, 8, 2, 128, max_kv_len=3 * PAGE, dtype=dtype, weights=True, **scales)
    for b, w, e in step(small, lens2, dec2, S.decode_workspace(dec2), acc2):
        assert w.shape[1] == budget + 1
    assert lens2.tolist() == [budget + 1] * 2


def cache_for_prefill(cache, inp):
    """The prefill's view of the grown cache: the same pages under its own table."""
    return S.PagedKV(cache.k_cache, cache.v_cache, torch.from_numpy(np.maximum(inp.block_table, 0)).cuda())
