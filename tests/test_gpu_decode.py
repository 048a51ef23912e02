"""stem_decode on the GPU against the float64 oracle: lengths from nothing to many pages,
head groups, drafted tokens, a shared prefix, collected weights, BF16 and FP8.  Everything
the operator must not use (unused slots, the rest of a last page) holds NaN."""
import math
import threading

import numpy as np
import pytest
import torch

from block_sparse_attention_oam_b200 import stem as S
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


class Setup:
    """A cache of NaN with the sequences' (and the prefix's) rows scattered over it."""

    def __init__(self, lens, Hq, Hkv, d, q_len=1, dtype="bf16", prefix=0, weights=False, max_kv_len=None, seed=0,
                 spread=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.prefix, self.n, self.Hq, self.Hkv, self.d = list(lens), prefix, q_len, Hq, Hkv, d
        B = len(self.lens)
        cap = max(self.lens + [1]) if max_kv_len is None else max_kv_len
        pages, pre = -(-cap // PAGE), -(-prefix // PAGE)
        slots = sum(-(-n // PAGE) for n in self.lens) + pre + 3
        perm = rng.permutation(slots).astype(np.int32)
        fp8 = dtype == "fp8_e4m3"
        self.scales = dict(q_scale=0.031, k_scale=0.02, v_scale=0.05) if fp8 else {}
        tt = torch.float8_e4m3fn if fp8 else torch.bfloat16

        def draw(*shape, scale=1.0, name="v_scale"):
            x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * scale)
            return (x / self.scales[name]).to(tt) if fp8 else x.to(tt)

        def value(x, name):
            return x.float().numpy().astype(np.float64) * self.scales.get(name, 1.0)

        kc = torch.full((slots, PAGE, Hkv, d), float("nan")).to(tt)
        vc = kc.clone()
        table = np.full((B, pages), 0, dtype=np.int32)
        at = pre
        raw = lambda x: x.view(torch.uint8 if fp8 else torch.int16)  # noqa: E731

        def place(slot_list, k, v):
            for p, slot in enumerate(slot_list):
                m = min(PAGE, k.shape[0] - p * PAGE)
                raw(kc)[slot, :m] = raw(k)[p * PAGE: p * PAGE + m]
                raw(vc)[slot, :m] = raw(v)[p * PAGE: p * PAGE + m]

        pk, pv = draw(prefix, Hkv, d, name="k_scale"), draw(prefix, Hkv, d)
        place(perm[:pre], pk, pv)
        self.kv = []
        for b, n in enumerate(self.lens):
            k, v = draw(n, Hkv, d, name="k_scale"), draw(n, Hkv, d)
            mine = perm[at: at + -(-n // PAGE)]
            at += len(mine)
            table[b, : len(mine)] = mine
            place(mine, k, v)
            self.kv.append((np.concatenate([value(pk, "k_scale"), value(k, "k_scale")]),
                            np.concatenate([value(pv, "v_scale"), value(v, "v_scale")])))
        q = draw(B * q_len, Hq, d, scale=spread, name="q_scale")
        self.qv = value(q, "q_scale")
        self.q = q.cuda()
        self.cache = S.PagedKV(kc.cuda(), vc.cuda(), torch.from_numpy(table).cuda())
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.prefix_table = torch.from_numpy(perm[:pre].copy()).cuda() if prefix else None
        self.dec = S.Decode(B, Hq, Hkv, d, max_kv_len=cap, q_len=q_len, dtype=dtype, prefix_len=prefix,
                            weights=weights, **self.scales)
        self.fp8, self.weights = fp8, weights
        self.lse = torch.full((Hq, B * q_len), 7.0, device="cuda")
        self.w_in = self.w_out = None
        if weights:
            stride = cap + 3                # any stride >= max_kv_len
            self.w_in = torch.rand((B, Hkv, stride), device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
            self.w_out = torch.full_like(self.w_in, -5.0)

    def call(self, **kw):
        kw = dict(prefix_table=self.prefix_table, weights_in=self.w_in, weights_out=self.w_out, lse=self.lse,
                  ws=S.decode_workspace(self.dec)) | kw
        out = S.stem_decode(self.dec, self.q, self.cache, self.kv_lens, **kw)
        assert S.query_status(kw["ws"]) == S.STEM_OK
        return out

    def check(self, out, lse=None):
        """Bounds by arithmetic.  A score is a sum of d products, added in float32 in at most
        d steps of relative 2^-22 (the matrix units may truncate): |ds| <= d 2^-22 sum|q k|;
        with the scaling, the exponential and the joining of partials (a few 2^-22 each)
        every weight is off by a relative e = d 2^-22 size + 2^-18 (1 + |lse|).  P is rounded
        to bf16 (2^-8) or, FP8, f16 (2^-11, and 2^-25 absolute below 2^-14 of weights whose
        largest is >= 1, each of the n keys).  O adds n products in float32 (n 2^-22) and is
        rounded to bf16 (2^-8 of its value)."""
        lse = self.lse if lse is None else lse
        got, got_lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        sigma, n = 1.0 / math.sqrt(self.d), self.n
        for b, (k, v) in enumerate(self.kv):
            rows = slice(b * n, b * n + n)
            ref, ref_lse, w, mean_abs, size = O.decode_rows(self.qv[rows], k, v, sigma, self.prefix)
            keys = k.shape[0]
            mag = np.where(np.isinf(ref_lse.T), 0.0, np.abs(ref_lse.T))
            e = self.d * 2.0 ** -22 * size + 2.0 ** -18 * (1 + mag)                    # [n, Hq]
            u = 2.0 ** -11 if self.fp8 else 2.0 ** -8
            vmax = np.abs(v).max() if keys else 0.0
            tiny = keys * 2.0 ** -25 * vmax if self.fp8 else 0.0
            bound = 2.0 ** -8 * np.abs(ref) + (u + 2 * e[..., None] + keys * 2.0 ** -22) * mean_abs * 1.01 + tiny + 1e-30
            err = np.abs(got[rows] - ref)
            assert np.isfinite(got[rows]).all(), f"sequence {b}"
            assert (err <= bound).all(), f"sequence {b}: {np.max(err / bound)} of the bound"
            g = got_lse[:, rows]
            assert np.array_equal(np.isinf(g), np.isinf(ref_lse)) and not np.isnan(g).any()
            fine = ~np.isinf(ref_lse)
            assert (np.abs(g[fine] - ref_lse[fine]) <= 2 * e.T[fine]).all()
            if self.weights:
                S_ = self.lens[b]
                was, now = (t[b].cpu().numpy().astype(np.float64) for t in (self.w_in, self.w_out))
                emax = e.max() if e.size else 0.0
                lim = 3 * emax * w + 2.0 ** -22 * (was[:, :S_] + w) + 1e-30
                assert (np.abs(now[:, :S_] - was[:, :S_] - w) <= lim).all(), f"weights of sequence {b}"
                assert (now[:, S_:] == -5.0).all(), f"sequence {b}: weights behind its last token were written"


LENS = [1, 0, 63, 64, 65, 128, 700]
CASES = {
    "one_token": dict(lens=[1], Hq=1, Hkv=1, d=64),
    "empty_batch": dict(lens=[0, 0], Hq=4, Hkv=2, d=128),
    "mha_d64": dict(lens=LENS, Hq=2, Hkv=2, d=64),
    "gqa4": dict(lens=LENS, Hq=8, Hkv=2, d=128),
    "gqa3_d64": dict(lens=LENS, Hq=9, Hkv=3, d=64),
    "gqa7": dict(lens=[500, 33], Hq=7, Hkv=1, d=128),
    "gqa16": dict(lens=[130, 64, 2], Hq=32, Hkv=2, d=128),
    "gqa17": dict(lens=[130, 64, 2], Hq=17, Hkv=1, d=64),
    "gqa40": dict(lens=[300, 1], Hq=40, Hkv=1, d=128),
    "long": dict(lens=[9000], Hq=4, Hkv=1, d=128),
    "long_many_partials": dict(lens=[20000, 3, 5000], Hq=8, Hkv=2, d=64),
    "big_scores": dict(lens=[700, 65], Hq=8, Hkv=2, d=128, spread=12.0),
    "q2": dict(lens=LENS, Hq=4, Hkv=2, d=64, q_len=2),
    "q5_gqa4": dict(lens=[3, 0, 5, 66, 700], Hq=8, Hkv=2, d=128, q_len=5),
    "q8_gqa3": dict(lens=[8, 71, 64, 128], Hq=6, Hkv=2, d=128, q_len=8),
    "q64": dict(lens=[64, 130, 30], Hq=2, Hkv=1, d=64, q_len=64),
    "fp8": dict(lens=LENS, Hq=8, Hkv=2, d=128, dtype="fp8_e4m3"),
    "fp8_q3_gqa5": dict(lens=[2, 3, 64, 66, 400], Hq=10, Hkv=2, d=128, q_len=3, dtype="fp8_e4m3"),
    "fp8_long": dict(lens=[9001, 20], Hq=8, Hkv=2, d=128, dtype="fp8_e4m3"),
    "prefix": dict(lens=LENS, Hq=8, Hkv=2, d=128, prefix=1000),
    "prefix_1": dict(lens=[1, 0, 5], Hq=2, Hkv=2, d=64, prefix=1),
    "prefix_64_q2": dict(lens=[2, 0, 1, 70], Hq=4, Hkv=1, d=128, prefix=64, q_len=2),
    "prefix_65_odd": dict(lens=[4, 9, 100], Hq=15, Hkv=3, d=64, prefix=65, q_len=3),
    "prefix_wide": dict(lens=[7] * 40 + [130], Hq=8, Hkv=2, d=128, prefix=2500),
    "prefix_wide_d64": dict(lens=[7] * 21 + [130], Hq=14, Hkv=2, d=64, prefix=1300),
    "prefix_wide_big": dict(lens=[7] * 70, Hq=4, Hkv=1, d=128, prefix=700, spread=12.0),
    "prefix_wide_q3": dict(lens=[7, 1, 0] * 15, Hq=10, Hkv=2, d=128, prefix=333, q_len=3),
    "prefix_fp8": dict(lens=[9, 64, 0], Hq=8, Hkv=2, d=128, prefix=300, dtype="fp8_e4m3"),
    "prefix_wide_fp8": dict(lens=[9, 64, 0] * 13, Hq=8, Hkv=2, d=128, prefix=1500, dtype="fp8_e4m3"),
    "weights": dict(lens=LENS, Hq=8, Hkv=2, d=128, weights=True),
    "weights_long": dict(lens=[20000, 1, 3000], Hq=4, Hkv=1, d=128, weights=True),
    "weights_q4_gqa5": dict(lens=[3, 4, 70, 500], Hq=10, Hkv=2, d=64, q_len=4, weights=True),
    "weights_rows300": dict(lens=[64, 200], Hq=10, Hkv=1, d=64, q_len=30, weights=True),
    "weights_fp8": dict(lens=LENS, Hq=8, Hkv=2, d=128, dtype="fp8_e4m3", weights=True),
    "weights_prefix": dict(lens=[5, 0, 130], Hq=8, Hkv=2, d=128, prefix=200, weights=True),
    "weights_prefix_wide": dict(lens=[5, 0, 130] * 9, Hq=8, Hkv=2, d=128, prefix=400, weights=True),
    "kv7": dict(lens=[130, 1, 64], Hq=7, Hkv=7, d=128),
    "kv11_q2": dict(lens=[130, 0, 65], Hq=22, Hkv=11, d=64, q_len=2),
    "kv5_fp8": dict(lens=[700, 9], Hq=5, Hkv=5, d=128, dtype="fp8_e4m3"),
    "gqa256_prefix": dict(lens=[3, 65], Hq=256, Hkv=1, d=64, prefix=70),
    "gqa128_prefix": dict(lens=[3, 65], Hq=128, Hkv=1, d=128, prefix=300),
    "gqa100_prefix": dict(lens=[3, 65, 0], Hq=100, Hkv=1, d=64, prefix=129),
    "gqa64_prefix_fp8": dict(lens=[9, 1, 20], Hq=64, Hkv=1, d=128, prefix=257, dtype="fp8_e4m3"),
    "prefix_wide_1": dict(lens=[1] * 50, Hq=2, Hkv=2, d=128, prefix=1),
    "prefix_wide_128": dict(lens=[2] * 20, Hq=8, Hkv=2, d=64, prefix=128),
    "prefix_wide_kv5": dict(lens=[5] * 30, Hq=20, Hkv=5, d=128, prefix=190),
    "prefix_wide_long": dict(lens=[3, 900] * 10, Hq=12, Hkv=2, d=128, prefix=9001),
    "prefix_wide_empty_own": dict(lens=[0] * 40, Hq=4, Hkv=2, d=64, prefix=100),
    "weights_prefix_wide_fp8": dict(lens=[70, 1] * 12, Hq=8, Hkv=2, d=128, prefix=200, q_len=2, dtype="fp8_e4m3", weights=True),
    "longest": dict(lens=[262144], Hq=1, Hkv=1, d=64),
    "most_sequences": dict(lens=[1 + b % 3 * 40 for b in range(1024)], Hq=2, Hkv=1, d=64),
    "bound_above_lengths": dict(lens=[5, 100], Hq=4, Hkv=2, d=64, max_kv_len=5000, weights=True),
}


@pytest.mark.parametrize("name", list(CASES))
def test_decode_matches_oracle(name):
    s = Setup(seed=sum(map(ord, name)), **CASES[name])
    s.check(s.call())


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "bf16"), (128, "fp8_e4m3")])
@pytest.mark.parametrize("prefix", [1, 63, 64, 65, 127, 128, 129, 192, 256, 257, 384, 640, 1500])
def test_prefix_lengths_around_its_tiles(d, dtype, prefix):
    """A wide batch over prefixes of a few tiles, with no own token and with a few."""
    s = Setup([0, 0, 3] * 14, Hq=8, Hkv=2, d=d, prefix=prefix, seed=prefix, dtype=dtype)
    s.check(s.call())


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "bf16"), (128, "fp8_e4m3")])
@pytest.mark.parametrize("prefix,cap", [(70, 1500), (1500, 1500), (70, 60000), (9001, 1500)])
def test_own_tokens_beside_the_prefix(d, dtype, prefix, cap):
    """Own tokens that outlast a wide batch's prefix, and a bound far above their number: both
    kernels at once, and more CTAs than find a place beside the prefix's."""
    s = Setup([0, 1500, 3, 64, 129] * 5, Hq=8, Hkv=2, d=d, prefix=prefix, seed=prefix + cap, dtype=dtype, max_kv_len=cap,
              weights=True)
    s.check(s.call())


def test_many_sequences():
    """More sequences than a CTA has threads, of every length."""
    rng = np.random.default_rng(3)
    s = Setup([int(x) for x in rng.integers(0, 200, 400)], Hq=2, Hkv=1, d=64, seed=9)
    s.check(s.call())


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_drafted_nan_rows_touch_later_rows_only(dtype):
    """A NaN in the newest token's K and V reaches that token's row and no earlier one."""
    s = Setup([70, 64, 15], Hq=8, Hkv=2, d=128, q_len=4, dtype=dtype, seed=5)
    clean = s.call().clone()
    for b, n in enumerate(s.lens):
        slot = int(s.cache.block_table[b, (n - 1) // PAGE])
        nan = torch.full((2, 128), float("nan"), device="cuda").to(s.q.dtype)
        for c in (s.cache.k_cache, s.cache.v_cache):
            c.view(torch.uint8)[slot, (n - 1) % PAGE] = nan.view(torch.uint8)
    out = s.call()
    for b in range(len(s.lens)):
        assert torch.equal(out[b * 4: b * 4 + 3], clean[b * 4: b * 4 + 3])
        assert torch.isnan(out[b * 4 + 3].float()).all()


def test_equal_calls_give_equal_bits_and_sequences_do_not_mix():
    s = Setup([3000, 1, 700, 0], Hq=8, Hkv=2, d=128, weights=True, seed=6)
    a = s.call().clone()
    w = s.w_out.clone()
    for _ in range(3):
        assert torch.equal(s.call(), a) and torch.equal(s.w_out, w)


def test_weights_in_place_and_without_input():
    s = Setup([300, 0, 65], Hq=8, Hkv=2, d=128, weights=True, seed=7)
    s.call()
    apart = s.w_out.clone()
    both = s.w_in.clone()
    s.call(weights_in=both, weights_out=both)
    for b, n in enumerate(s.lens):
        assert torch.equal(both[b, :, :n], apart[b, :, :n])
        assert torch.equal(both[b, :, n:], s.w_in[b, :, n:])
    fresh = torch.full_like(both, -5.0)
    s.call(weights_in=None, weights_out=fresh)
    for b, n in enumerate(s.lens):
        # float32 addition of the same sums: half a step of a value below 2, twice
        assert torch.allclose(fresh[b, :, :n] + s.w_in[b, :, :n], apart[b, :, :n], rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("prefix,more", [(0, 0), (500, 0), (500, 20)])
def test_captured_step_follows_the_lengths(prefix, more):
    """A captured step replayed as the sequences grow equals the call made anew."""
    s = Setup([700, 130, 64] + [5] * more, Hq=8, Hkv=2, d=128, prefix=prefix, weights=True, seed=8)
    ws = S.decode_workspace(s.dec)
    out = torch.empty((3 + more, 8, 128), dtype=torch.bfloat16, device="cuda")
    s.call(out=out, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.stem_decode(s.dec, s.q, s.cache, s.kv_lens, prefix_table=s.prefix_table, weights_in=s.w_in,
                      weights_out=s.w_out, out=out, lse=s.lse, ws=ws)
    full = list(s.lens)
    for lens in ([1, 1, 1], [65, 0, 64], [699, 129, 3], full):
        s.kv_lens[:3] = torch.tensor(lens[:3], dtype=torch.int32)
        s.w_out.fill_(-5.0)
        g.replay()
        got, got_lse, got_w = out.clone(), s.lse.clone(), s.w_out.clone()
        s.w_out.fill_(-5.0)
        assert torch.equal(s.call(), got)
        assert torch.equal(s.lse, got_lse) and torch.equal(s.w_out, got_w)


def test_two_streams_with_their_own_workspaces():
    a = Setup([9000, 40], Hq=8, Hkv=2, d=128, seed=10)
    b = Setup([5000, 600], Hq=8, Hkv=2, d=128, seed=11)
    wa, wb = S.decode_workspace(a.dec), S.decode_workspace(b.dec)
    ra, rb = a.call(ws=wa).clone(), b.call(ws=wb).clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs.append((S.stem_decode(a.dec, a.q, a.cache, a.kv_lens, out=torch.empty_like(ra), ws=wa, stream=s1),
                     S.stem_decode(b.dec, b.q, b.cache, b.kv_lens, out=torch.empty_like(rb), ws=wb, stream=s2)))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, ra) and torch.equal(y, rb)


def test_threads_on_streams_of_their_own():
    """Python threads that call at once, wide batches behind a prefix among them (the prefix's
    kernel and decode_kernel side by side, twice), get what a call alone gets."""
    kinds = [dict(lens=[30, 700] * 20, prefix=2000), dict(lens=[3] * 41, prefix=5000), dict(lens=[900, 0, 77], prefix=0)]
    sets = [Setup(Hq=8, Hkv=2, d=128, seed=30 + i, **k) for i, k in enumerate(kinds)]
    wss = [S.decode_workspace(s.dec) for s in sets]
    alone = [s.call(ws=w).clone() for s, w in zip(sets, wss)]
    outs = [[torch.empty_like(r) for _ in range(20)] for r in alone]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for o in outs[i]:
                    s = sets[i]
                    S.stem_decode(s.dec, s.q, s.cache, s.kv_lens, prefix_table=s.prefix_table, out=o, ws=wss[i])
        except Exception as e:  # noqa: BLE001  (shown by the assertion)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i, r in enumerate(alone):
        assert all(torch.equal(o, r) for o in outs[i])


@pytest.mark.parametrize("name", ["gqa4", "q5_gqa4", "prefix_wide", "prefix_wide_fp8", "weights_q4_gqa5", "weights_fp8"])
def test_writes_only_its_buffers(name):
    s = Setup(seed=21, **CASES[name])
    rows = len(s.lens) * s.n
    out, lse = Guarded((rows, s.Hq, s.d), torch.bfloat16), Guarded((s.Hq, rows), torch.float32)
    ws = Guarded((s.dec.workspace_bytes(),), torch.uint8)
    ws.t.zero_()
    snap = [t.clone() for t in (s.cache.k_cache.view(torch.uint8), s.cache.v_cache.view(torch.uint8), s.cache.block_table, s.q.view(torch.uint8), s.kv_lens)]
    w = None
    if s.weights:
        w = Guarded(tuple(s.w_out.shape), torch.float32)
        w.t.fill_(-5.0)
        s.w_out = w.t
    s.check(s.call(out=out.t, lse=lse.t, ws=ws.t), lse.t)
    for g in (out, lse, ws, w):
        assert g is None or g.intact()
    for x, y in zip(snap, (s.cache.k_cache.view(torch.uint8), s.cache.v_cache.view(torch.uint8), s.cache.block_table, s.q.view(torch.uint8), s.kv_lens)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("prefix", [0, 200])
def test_what_follows_in_the_stream_sees_the_result(prefix):
    """Calls, copies of their outputs and changes of their inputs in one stream, nothing
    waited for in between (short sequences: no row is shared by two CTAs)."""
    s = Setup([9, 64, 1, 30] * 20, Hq=8, Hkv=2, d=128, prefix=prefix, seed=14)
    ws = S.decode_workspace(s.dec)
    q0 = s.q.clone()
    qs = [q0.roll(i, 0).contiguous() for i in range(6)]
    want = []
    for q in qs:
        s.q.copy_(q)
        want.append(s.call(ws=ws).clone())
        torch.cuda.synchronize()
    out, got = torch.empty_like(want[0]), []
    for _ in range(3):
        for q in qs:
            s.q.copy_(q)
            S.stem_decode(s.dec, s.q, s.cache, s.kv_lens, prefix_table=s.prefix_table, out=out, ws=ws)
            got.append(out.clone())
            out.zero_()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 6]), i


def test_pages_beyond_32_bit_offsets():
    """Pages at the far end of a cache of more than 4 GB (per tensor) give what the same rows
    give in a small one, through the own and the prefix path, and moved by an eviction."""
    s = Setup([130, 64] + [7] * 20, Hq=32, Hkv=8, d=128, prefix=100, seed=15)
    want = s.call().clone()
    slots = 36000
    assert slots * PAGE * 8 * 128 * 2 > 1 << 32
    near = s.cache.k_cache.shape[0]
    k = torch.empty((slots, PAGE, 8, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[slots - near:].copy_(s.cache.k_cache)
    v[slots - near:].copy_(s.cache.v_cache)
    far = slots - near
    cache = S.PagedKV(k, v, s.cache.block_table + far)
    out = S.stem_decode(s.dec, s.q, cache, s.kv_lens, prefix_table=s.prefix_table + far, lse=s.lse)
    assert torch.equal(out, want)
    w = torch.rand((22, 8, 192), device="cuda")
    ev = S.Evict(22, 8, 128, max_kv_len=130, budget=50, recent=5)
    fresh = torch.arange(22, dtype=torch.int32, device="cuda")[:, None].contiguous()
    small = S.PagedKV(torch.zeros((22, PAGE, 8, 128), dtype=torch.bfloat16, device="cuda"),
                      torch.zeros((22, PAGE, 8, 128), dtype=torch.bfloat16, device="cuda"), fresh)
    keep, lens = S.stem_evict(ev, s.cache, s.kv_lens, w, small)
    keep2, lens2 = S.stem_evict(ev, cache, s.kv_lens, w, S.PagedKV(k, v, fresh + (far - 22)))
    assert torch.equal(keep, keep2) and torch.equal(lens, lens2)
    for b, n in enumerate(lens.tolist()):
        assert torch.equal(k[far - 22 + b, :n].view(torch.int16), small.k_cache[b, :n].view(torch.int16))
        assert torch.equal(v[far - 22 + b, :n].view(torch.int16), small.v_cache[b, :n].view(torch.int16))


def test_two_graphs_take_turns_on_one_workspace():
    """Two captured problems of other shapes that share a workspace, replayed in turn."""
    a = Setup([3000, 64], Hq=8, Hkv=2, d=128, seed=16)
    b = Setup([65, 9, 700] * 8, Hq=8, Hkv=2, d=64, prefix=130, weights=True, seed=17)
    ws = torch.zeros(max(a.dec.workspace_bytes(), b.dec.workspace_bytes()), dtype=torch.uint8, device="cuda")
    outs, graphs, want = [], [], []
    for s in (a, b):
        want.append(s.call(ws=ws).clone())
        out = torch.empty_like(want[-1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.stem_decode(s.dec, s.q, s.cache, s.kv_lens, prefix_table=s.prefix_table, weights_in=s.w_in, weights_out=s.w_out, out=out, ws=ws)
        outs.append(out)
        graphs.append(g)
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.parametrize("name", ["q", "cache.k_cache", "cache.v_cache", "cache.block_table", "kv_lens", "prefix_table",
                                  "weights_in", "weights_out", "out", "lse", "ws"])
def test_tensors_that_do_not_fit_are_named(name):
    """Another type, another shape, strides, and host memory: refused before anything runs."""
    s = Setup([5, 70], Hq=8, Hkv=2, d=128, prefix=100, weights=True)
    out = torch.full_like(s.q, 7.0)
    ws = S.decode_workspace(s.dec)
    args = {"q": s.q, "cache.k_cache": s.cache.k_cache, "cache.v_cache": s.cache.v_cache, "cache.block_table": s.cache.block_table,
            "kv_lens": s.kv_lens, "prefix_table": s.prefix_table, "weights_in": s.w_in, "weights_out": s.w_out, "out": out,
            "lse": s.lse, "ws": ws}

    def call(**kw):
        x = args | kw
        return S.stem_decode(s.dec, x["q"], S.PagedKV(x["cache.k_cache"], x["cache.v_cache"], x["cache.block_table"]),
                             x["kv_lens"], prefix_table=x["prefix_table"], weights_in=x["weights_in"],
                             weights_out=x["weights_out"], out=x["out"], lse=x["lse"], ws=x["ws"])

    t = args[name]
    wide = torch.zeros((*t.shape, 2), dtype=t.dtype, device=t.device)
    with pytest.raises((ValueError, S.StemError)):  # no width: some of these the library itself refuses
        call(**{name: t[..., :0]})
    for x in (t.cpu(), t.to(torch.float64), wide[..., 0], wide):
        if name == "q" and not x.is_cuda:
            with pytest.raises(ValueError):
                call(**{name: x})
        else:
            with pytest.raises(ValueError, match=name.replace(".", "[.]") if name != "cache.k_cache" else "cache[.]"):
                call(**{name: x})
    torch.cuda.synchronize()
    assert (out == 7).all()


def test_bad_pages_and_lengths_are_reported():
    """A page outside the cache is read as slot 0, a length outside [0, max_kv_len] is
    clamped; both are reported, and the sequences beside them are right."""
    s = Setup([130, 64], Hq=4, Hkv=2, d=64, seed=12)
    want = s.call().clone()
    for bad in (-1, s.cache.k_cache.shape[0], 1 << 30):
        table = s.cache.block_table.clone()
        table[0, 1] = bad
        ws = S.decode_workspace(s.dec)
        out = S.stem_decode(s.dec, s.q, S.PagedKV(s.cache.k_cache, s.cache.v_cache, table), s.kv_lens, ws=ws)
        with pytest.raises(S.StemError) as e:
            S.query_status(ws)
        assert e.value.status == S.STEM_ERR_BOUNDS
        assert torch.equal(out[1], want[1])
    for bad in (-1, 131):
        lens = s.kv_lens.clone()
        lens[0] = bad
        ws = S.decode_workspace(s.dec)
        out = S.stem_decode(s.dec, s.q, s.cache, lens, ws=ws)
        with pytest.raises(S.StemError) as e:
            S.query_status(ws)
        assert e.value.status == S.STEM_ERR_BOUNDS
        assert torch.equal(out[1], want[1])
        assert torch.equal(out[0], torch.zeros_like(out[0]) if bad < 0 else want[0])


def test_last_row_of_a_dense_prefill():
    """The newest token over the cache of a prefill equals the prefill's own last row (both
    round P to bf16: twice the oracle bound of one)."""
    from block_sparse_attention_oam_b200 import workloads as W
    wl = W.PAGED_VARLEN.with_(name="decode_after_prefill", seqlens=(1024, 300), num_q_heads=8, num_kv_heads=2, seed=31)
    inp = W.make_inputs(wl)
    prob = S.problem_for(wl, inp)
    cache = S.PagedKV(inp.k_cache.cuda(), inp.v_cache.cuda(), torch.from_numpy(inp.block_table).cuda())
    q = inp.q.cuda()
    dense = S.bsa_dense_prefill(prob, q, q, q, paged=cache)
    last = torch.tensor([1023, 1323], device="cuda")
    dec = S.Decode(2, 8, 2, 128, max_kv_len=1024)
    lens = torch.tensor([1024, 300], dtype=torch.int32, device="cuda")
    out = S.stem_decode(dec, q[last].contiguous(), cache, lens)
    v = np.abs(inp.dequant("v"))
    bound = 2 * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -12) * v.max()
    assert (out.float() - dense[last].float()).abs().max().item() <= bound
    assert out.float().abs().max().item() > 0
