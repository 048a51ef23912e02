"""stem_decode's numbers where they are hardest to hold: a long even tail under one dominant key,
and sequences beside one that holds huge values and NaN."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_oam_b200 import stem as S
from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu

PAGE = S.PAGE_SIZE


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


# One key of weight 1 and value 0, then n - 1 keys of weight 2^-x and value v: together they make
# the output.  Enough rows that one CTA sees all of a row's keys against that one maximum: 444
# sequences for decode_kernel's CTAs, 96 units of 256 rows for prefix_kernel's.
TAILS = {
    "own_128k": dict(B=444, n=1, own=131072, prefix=0),
    "own_256k": dict(B=444, n=1, own=262144, prefix=0),
    "prefix_128k": dict(B=512, n=48, own=48, prefix=131072),
    "prefix_256k": dict(B=512, n=48, own=48, prefix=262144),
}


@pytest.mark.parametrize("below", [24.5, 25.5, 27.0])
@pytest.mark.parametrize("name", list(TAILS))
def test_a_long_tail_under_a_dominant_key(name, below):
    """FP8, where P is held in f16.  Bound: as in the decode tests' check(), P's rounding (2^-11
    of each key's weight), the statistics' error e, sums over n keys (n 2^-22, O's and l's) and
    the output's bf16 (2^-8); and for what f16 holds below its normal range, half a step of 2^-24
    where the largest entry is at least 2^7: 2^-32 of the largest weight a key."""
    c = TAILS[name]
    B, n, d = c["B"], c["n"], 128
    keys = c["prefix"] or c["own"]
    # scores (log2): 0 for the first key, -below for the others.  q = (8, 0 ...), k = (code, 0 ...):
    # sigma * log2(e) * 8 * q_scale * k_scale * (448 - code) = below, codes 448 and -448
    scale = below / (math.log2(math.e) / math.sqrt(d) * 8 * 896)
    e4 = torch.float8_e4m3fn
    k = torch.zeros((4, PAGE, 1, d))
    v = torch.zeros((4, PAGE, 1, d))
    k[..., 0] = -448.0
    k[0, 0, 0, 0] = 448.0
    v[..., :] = 256.0
    v[0, 0] = 0.0
    k[2], v[2] = float("nan"), float("nan")          # the new tokens behind a prefix; the first of a row's own is its last
    table = torch.ones((B, -(-c["own"] // PAGE)), dtype=torch.int32)
    prefix_table = None
    if c["prefix"]:
        prefix_table = torch.ones(c["prefix"] // PAGE, dtype=torch.int32)
        prefix_table[0] = 0
        prefix_table = prefix_table.cuda()
        lens = torch.zeros(B, dtype=torch.int32)     # nothing of their own
        table[:] = 2
    else:
        table[:, 0] = 0
        lens = torch.full((B,), c["own"], dtype=torch.int32)
    q = torch.zeros((B * n, 1, d))
    q[..., 0] = 8.0
    dec = S.Decode(B, 1, 1, d, max_kv_len=c["own"], q_len=n, dtype="fp8_e4m3", q_scale=1.0, k_scale=scale, v_scale=0.5, prefix_len=c["prefix"])
    lse = torch.zeros((1, B * n), device="cuda")
    out = S.stem_decode(dec, q.to(e4).cuda(), S.PagedKV(k.to(e4).cuda(), v.to(e4).cuda(), table.cuda()), lens.cuda(),
                        prefix_table=prefix_table, lse=lse)
    gap = float(np.float32(scale)) * 8 * 896 / math.sqrt(d) * math.log2(math.e)
    tail = (keys - 1) * 2.0 ** -gap
    ref = 128.0 * tail / (1 + tail)
    top = float(np.float32(scale)) * 8 * 448 / math.sqrt(d)
    e = d * 2.0 ** -22 * top + 2.0 ** -18 * (1 + top)
    tiny = keys * 2.0 ** -32 * 128.0 / (1 + tail)
    bound = 2.0 ** -8 * ref + (2.0 ** -11 + 2 * e + keys * 2.0 ** -22) * ref * 1.01 + tiny
    err = (out.double() - ref).abs().max().item()
    assert err <= bound, f"{err} against {bound}, of {ref}"
    ref_lse = top + math.log1p(tail)
    assert (lse.double() - ref_lse).abs().max().item() <= 2 * e


@pytest.mark.parametrize("v_scale", [1.6e-39, 1e35])
@pytest.mark.parametrize("B,prefix", [(1, 0), (500, 0), (60, 65001)])
def test_value_scales_at_the_ends_of_float32(v_scale, B, prefix):
    """A mean of 64K equal values, joined from many CTAs' shares or within one: all operations
    between are relative errors of 2^-20 at most, the output's rounding 2^-8."""
    table = torch.zeros((B, 1024), dtype=torch.int32, device="cuda")
    e4 = torch.float8_e4m3fn
    kv = S.PagedKV(torch.zeros((1, PAGE, 1, 128), device="cuda").to(e4), torch.full((1, PAGE, 1, 128), 8.0, device="cuda").to(e4), table)
    dec = S.Decode(B, 1, 1, 128, max_kv_len=65536, dtype="fp8_e4m3", v_scale=v_scale, prefix_len=prefix)
    lens = torch.full((B,), 0 if prefix else 65536, dtype=torch.int32, device="cuda")
    ptable = torch.zeros(-(-prefix // PAGE), dtype=torch.int32, device="cuda") if prefix else None
    out = S.stem_decode(dec, torch.ones((B, 1, 128), device="cuda").to(e4), kv, lens, prefix_table=ptable)
    want = 8 * float(np.float32(v_scale))
    assert ((out.double() / want - 1).abs() <= 2.0 ** -8 * 1.01).all()


GROUPS = {
    "own": dict(lens=[300, 65, 700, 9], Hq=8, Hkv=2, d=128, weights=True),
    "own_q3": dict(lens=[300, 65, 700, 9], Hq=8, Hkv=2, d=128, q_len=3),
    "narrow_prefix": dict(lens=[30, 65, 0, 9], Hq=8, Hkv=2, d=128, prefix=1000, weights=True),
    "narrow_prefix_d64": dict(lens=[30, 65, 0, 9], Hq=8, Hkv=2, d=64, prefix=1000),
    "narrow_prefix_fp8": dict(lens=[30, 65, 0, 9], Hq=8, Hkv=2, d=128, prefix=1000, dtype="fp8_e4m3"),
    "wide_prefix": dict(lens=[30, 65, 0, 9] * 10, Hq=8, Hkv=2, d=128, prefix=1000, weights=True),
    "wide_prefix_fp8": dict(lens=[30, 65, 0, 9] * 10, Hq=8, Hkv=2, d=128, prefix=1000, dtype="fp8_e4m3"),
}


@pytest.mark.parametrize("hold", ["large", "nan"])
@pytest.mark.parametrize("name", list(GROUPS))
def test_a_sequence_leaves_the_others_alone(name, hold):
    """Other queries, keys and values of one sequence, the lengths as they were (so that the work
    is split as before): every other sequence's output, log-sum-exp and weights keep their bits."""
    s = D.Setup(seed=60, **GROUPS[name])
    ws = S.decode_workspace(s.dec)
    want = s.call(ws=ws).clone()
    want_lse, want_w = s.lse.clone(), s.w_out.clone() if s.weights else None
    changed = 1
    x = torch.full((s.d,), float("nan") if hold == "nan" else 400.0, device="cuda").to(s.q.dtype).view(torch.uint8)
    s.q.view(torch.uint8)[changed * s.n: (changed + 1) * s.n] = x
    n = s.lens[changed]
    for p in range(-(-n // PAGE)):
        slot = int(s.cache.block_table[changed, p])
        for c in (s.cache.k_cache, s.cache.v_cache):
            c.view(torch.uint8)[slot, : min(PAGE, n - p * PAGE)] = x
    got = s.call(ws=ws)
    rows = [r for r in range(len(s.lens) * s.n) if r // s.n != changed]
    assert torch.equal(got[rows], want[rows])
    assert torch.equal(s.lse[:, rows], want_lse[:, rows])
    if s.weights:
        others = [b for b in range(len(s.lens)) if b != changed]
        assert torch.equal(s.w_out[others], want_w[others])
    assert not torch.equal(got[changed * s.n: (changed + 1) * s.n], want[changed * s.n: (changed + 1) * s.n])
