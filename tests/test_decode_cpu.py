"""Decoding operators without a GPU: every refusal happens on the host before any CUDA
call, workspace sizes follow the problem, and the oracle's rows and eviction rule are
pinned by hand."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from block_sparse_attention_oam_b200 import build as B
from block_sparse_attention_oam_b200 import stem as S
from oracle import stem_oracle as O


@pytest.fixture(scope="module")
def L():
    B.build()
    return S.lib()


FAKE = ctypes.c_void_p(0x1000)      # never dereferenced: validation fails first
GOOD = dict(num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=128, max_kv_len=1000)


def paged(max_pages=16, slots=64, page=64, k=0x1000, v=0x1000, table=0x1000):
    return S._Paged(k, v, table, page, max_pages, slots)


def decode(L, dec, q=FAKE, cache=None, lens=FAKE, ptable=None, w_in=None, w_out=None, stride=0, out=FAKE, ws=FAKE,
           ws_bytes=1 << 40):
    cache = paged() if cache is None else cache
    return L.stem_decode(dec.c, q, ctypes.byref(cache) if cache else None, lens, ptable, w_in, w_out, stride, out,
                         None, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(num_seqs=0), S.STEM_ERR_INVALID),
    (dict(num_seqs=1025), S.STEM_ERR_INVALID),
    (dict(num_q_heads=7), S.STEM_ERR_INVALID),
    (dict(num_q_heads=0), S.STEM_ERR_INVALID),
    (dict(num_kv_heads=0), S.STEM_ERR_INVALID),
    (dict(num_q_heads=258), S.STEM_ERR_UNSUPPORTED),
    (dict(head_dim=96), S.STEM_ERR_UNSUPPORTED),
    (dict(head_dim=64, dtype="fp8_e4m3"), S.STEM_ERR_UNSUPPORTED),
    (dict(q_len=0), S.STEM_ERR_INVALID),
    (dict(q_len=65), S.STEM_ERR_INVALID),
    (dict(max_kv_len=0), S.STEM_ERR_INVALID),
    (dict(max_kv_len=262145), S.STEM_ERR_INVALID),
    (dict(prefix_len=-1), S.STEM_ERR_INVALID),
    (dict(prefix_len=262145), S.STEM_ERR_INVALID),
    (dict(dtype="fp8_e4m3", k_scale=0.0), S.STEM_ERR_INVALID),
    (dict(dtype="fp8_e4m3", v_scale=float("nan")), S.STEM_ERR_INVALID),
    (dict(softmax_scale=float("inf")), S.STEM_ERR_INVALID),
    (dict(num_seqs=1024, num_q_heads=256, num_kv_heads=256, max_kv_len=262144, q_len=64), S.STEM_ERR_UNSUPPORTED),
])
def test_decode_refuses_bad_problems(L, change, status):
    dec = S.Decode(**(GOOD | change))
    assert decode(L, dec, cache=paged(max_pages=1 << 20)) == status
    assert L.stem_decode_workspace_size(dec.c) == 0
    with pytest.raises(S.StemError):
        dec.workspace_bytes()


def test_decode_refuses_bad_buffers(L):
    dec = S.Decode(**GOOD)
    odd = ctypes.c_void_p(0x1008)
    assert L.stem_decode(None, FAKE, ctypes.byref(paged()), FAKE, None, None, None, 0, FAKE, None, FAKE, 1 << 40, None) == S.STEM_ERR_INVALID
    assert decode(L, dec, cache=False) == S.STEM_ERR_INVALID
    assert decode(L, dec, q=None) == S.STEM_ERR_INVALID
    assert decode(L, dec, q=odd) == S.STEM_ERR_INVALID
    assert decode(L, dec, out=None) == S.STEM_ERR_INVALID
    assert decode(L, dec, out=odd) == S.STEM_ERR_INVALID
    assert decode(L, dec, lens=None) == S.STEM_ERR_INVALID
    assert decode(L, dec, cache=paged(k=0)) == S.STEM_ERR_INVALID
    assert decode(L, dec, cache=paged(v=0x1004)) == S.STEM_ERR_INVALID
    assert decode(L, dec, cache=paged(page=32)) == S.STEM_ERR_UNSUPPORTED
    assert decode(L, dec, cache=paged(max_pages=15)) == S.STEM_ERR_INVALID
    assert decode(L, dec, cache=paged(slots=0)) == S.STEM_ERR_INVALID
    assert decode(L, dec, ptable=FAKE) == S.STEM_ERR_INVALID                      # no prefix
    assert decode(L, S.Decode(**GOOD, prefix_len=5)) == S.STEM_ERR_INVALID        # no prefix pages
    assert decode(L, dec, w_out=FAKE, stride=1000) == S.STEM_ERR_INVALID          # weights not asked for
    w = S.Decode(**GOOD, weights=True)
    assert decode(L, w) == S.STEM_ERR_INVALID
    assert decode(L, w, w_out=FAKE, stride=999) == S.STEM_ERR_INVALID
    assert decode(L, w, w_out=FAKE, w_in=ctypes.c_void_p(0x1010), stride=1000) == S.STEM_ERR_INVALID
    assert b"overlap" in L.stem_last_error()
    assert decode(L, dec, ws=None) == S.STEM_ERR_WORKSPACE
    assert decode(L, dec, ws=ctypes.c_void_p(0x1010)) == S.STEM_ERR_WORKSPACE
    assert decode(L, dec, ws_bytes=dec.workspace_bytes() - 1) == S.STEM_ERR_WORKSPACE


def test_decode_workspace_grows_with_the_problem(L):
    base = S.Decode(**GOOD).workspace_bytes()
    assert S.Decode(**(GOOD | dict(num_seqs=30))).workspace_bytes() > base
    assert S.Decode(**GOOD, prefix_len=100).workspace_bytes() > base
    # scores of every row and cached token, in float32
    assert S.Decode(**GOOD, weights=True).workspace_bytes() >= base + 3 * 8 * 1024 * 4


def test_decode_binding_checks_tensors(L):
    dec = S.Decode(**GOOD)
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    cache = S.PagedKV(torch.zeros((4, 64, 2, 128), dtype=torch.bfloat16), torch.zeros((4, 64, 2, 128), dtype=torch.bfloat16), torch.zeros((3, 16), dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        S.stem_decode(dec, q, cache, torch.zeros(3, dtype=torch.int32))
    dev = q.device
    with pytest.raises(ValueError, match="q must be"):
        S._tensor("q", q[:, ::2], (3, 4, 128), torch.bfloat16, dev)
    with pytest.raises(ValueError, match="q must be"):
        S._tensor("q", q, (3, 8, 64), torch.bfloat16, dev)
    with pytest.raises(ValueError, match="q must be"):
        S._tensor("q", q.float(), (3, 8, 128), torch.bfloat16, dev)
    with pytest.raises(ValueError, match="block_table"):
        S._pages("cache", cache, 4, 2, 128, torch.bfloat16, dev)
    with pytest.raises(ValueError, match="dtype"):
        S.Decode(**GOOD, dtype="fp16")


def test_native_entries_refuse_without_a_call(L):
    """Host tensors, other things than tensors, a wrong problem or a wrong number of arguments
    never reach the library (whose entry point is given as an address that holds no code)."""
    decode, _, evict, _ = S._binding()
    dec, ev = S.Decode(**GOOD), S.Evict(3, 2, 128, 1024, 64)
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    k, table, lens = torch.zeros((4, 64, 2, 128), dtype=torch.bfloat16), torch.zeros((3, 16), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    rest = (k, k, table, lens, None, None, None, q, None, torch.zeros(8, dtype=torch.uint8), None)
    assert decode(8, dec._c, q, *rest) == -1
    assert decode(8, dec._c, None, *rest) == -1
    w, ws = torch.zeros(3, 2, 1024), torch.zeros(8, dtype=torch.uint8)
    rest_e = (k, k, table, k, k, table, lens, lens, None, torch.zeros((3, 2, 64), dtype=torch.int32), ws, None)
    assert evict(8, ev._c, w, *rest_e) == -1
    assert evict(8, ev._c, w[0], *rest_e) == -1
    with pytest.raises(ValueError):
        decode(0, dec._c, q, *rest)
    with pytest.raises(ValueError):
        decode(8, ev._c, q, *rest)
    with pytest.raises(TypeError):
        decode(8, dec, q, *rest)
    with pytest.raises(TypeError):
        decode(8, dec._c, q)
    with pytest.raises(TypeError):
        evict(8, ev._c)


PROGRAM = r"""
#include <stdio.h>
#include "stem.h"
int main(void) {
  stem_decode_t d = {0};
  stem_evict_t e = {0};
  stem_paged_kv_t none = {0};
  d.num_seqs = 3; d.q_len = 1; d.num_q_heads = 8; d.num_kv_heads = 2; d.head_dim = 128; d.dtype = STEM_DT_BF16;
  d.max_kv_len = 1000;
  e.num_seqs = 3; e.num_kv_heads = 2; e.head_dim = 128; e.dtype = STEM_DT_BF16; e.max_kv_len = 1000; e.budget = 100;
  if (stem_decode(&d, 0, &none, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != STEM_ERR_INVALID) return 10;
  if (stem_evict(&e, &none, 0, 0, 0, &none, 0, 0, 0, 0, 0, 0, 0) != STEM_ERR_INVALID) return 11;
  if (stem_last_error()[0] == 0) return 12;
  printf("%zu %zu\n", stem_decode_workspace_size(&d), stem_evict_workspace_size(&e));
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_decoding_entry_points_from_c99(L, tmp_path):
    """A C99 program links the decoding entry points and gets the sizes the binding gets."""
    lib_dir = os.path.dirname(S.LIB_PATH)
    src, exe = tmp_path / "d.c", tmp_path / "d"
    src.write_text(PROGRAM)
    cc = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", str(src), "-I",
                         os.path.dirname(S.HEADER), "-L", lib_dir, "-lstem", "-Wl,-rpath," + lib_dir, "-o", str(exe)],
                        capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, (run.returncode, run.stdout, run.stderr)
    assert run.stdout.split() == [str(S.Decode(**GOOD).workspace_bytes()), "256"]


def test_library_exports_the_decoding_entry_points(L):
    names = S.header_functions()
    for n in ("stem_decode", "stem_decode_workspace_size", "stem_evict", "stem_evict_workspace_size"):
        assert n in names and hasattr(L, n)


def test_oracle_decode_rows_by_hand():
    """Two keys of equal score: the mean of their values; a row that sees one key, that value;
    a row that sees nothing, zero."""
    q = np.ones((3, 1, 2))
    k = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    v = np.array([[[2.0, 0.0]], [[4.0, 6.0]]])
    out, lse, w, _, _ = O.decode_rows(q, k, v, 1.0)
    assert np.allclose(out[:, 0], [[0, 0], [2, 0], [3, 3]])
    assert np.isneginf(lse[0, 0]) and np.allclose(lse[0, 1:], [1.0, 1.0 + np.log(2)])
    assert np.allclose(w, [[1.5, 0.5]])
    # the same two keys, the first as a shared prefix: every row sees it
    out, lse, w, _, _ = O.decode_rows(q[:2], k, v, 1.0, prefix=1)
    assert np.allclose(out[:, 0], [[2, 0], [3, 3]]) and np.allclose(w, [[0.5]])


def test_oracle_agrees_with_its_own_prefill():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((100, 4, 8)), rng.standard_normal((100, 2, 8)), rng.standard_normal((100, 2, 8))
    lists = [[[0, 1][: i + 1] for i in range(2)] for _ in range(4)]
    out, lse = O.attend(q, k, v, lists, 64, 0.3)
    got, got_lse, w, _, _ = O.decode_rows(q[97:], k, v, 0.3)
    assert np.allclose(got, out[97:]) and np.allclose(got_lse, lse[:, 97:])
    assert np.allclose(w.sum(1), 3 * 2)          # every row's weights add up to one


EV = dict(num_seqs=3, num_kv_heads=2, head_dim=128, max_kv_len=1000, budget=100)


def evict(L, ev, src=None, dst=None, lens=0x1000, w=0x100000, stride=1000, lens_out=0x2000, w_out=None, stride_out=0,
          keep=0x1000, ws=0x1000, ws_bytes=256):
    src = paged() if src is None else src
    dst = paged(max_pages=2) if dst is None else dst
    return L.stem_evict(ev.c, ctypes.byref(src) if src else None, lens, w, stride, ctypes.byref(dst) if dst else None,
                        lens_out, w_out, stride_out, keep, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(num_seqs=0), S.STEM_ERR_INVALID),
    (dict(num_seqs=1025), S.STEM_ERR_INVALID),
    (dict(num_kv_heads=0), S.STEM_ERR_INVALID),
    (dict(num_kv_heads=257), S.STEM_ERR_INVALID),
    (dict(head_dim=80), S.STEM_ERR_UNSUPPORTED),
    (dict(head_dim=64, dtype="fp8_e4m3"), S.STEM_ERR_UNSUPPORTED),
    (dict(max_kv_len=0), S.STEM_ERR_INVALID),
    (dict(budget=0), S.STEM_ERR_INVALID),
    (dict(budget=262145), S.STEM_ERR_INVALID),
    (dict(sink=-1), S.STEM_ERR_INVALID),
    (dict(recent=-1), S.STEM_ERR_INVALID),
    (dict(sink=60, recent=41), S.STEM_ERR_INVALID),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), S.STEM_ERR_INVALID),
])
def test_evict_refuses_bad_problems(L, change, status):
    ev = S.Evict(**(EV | change))
    assert evict(L, ev) == status
    assert L.stem_evict_workspace_size(ev.c) == 0
    with pytest.raises(S.StemError):
        ev.workspace_bytes()


def test_evict_refuses_bad_buffers(L):
    ev = S.Evict(**EV)
    for kw in (dict(src=False), dict(dst=False), dict(lens=None), dict(w=None), dict(lens_out=None), dict(keep=None),
               dict(stride=999), dict(lens_out=0x1000), dict(lens_out=0x1008), dict(src=paged(max_pages=15)),
               dict(dst=paged(max_pages=1)), dict(dst=paged(k=0x1008)), dict(w_out=0x200000, stride_out=99),
               dict(w_out=0x100010, stride_out=100)):
        assert evict(L, ev, **kw) == S.STEM_ERR_INVALID, kw
    assert evict(L, ev, src=paged(page=16)) == S.STEM_ERR_UNSUPPORTED
    assert evict(L, ev, ws=None) == S.STEM_ERR_WORKSPACE
    assert evict(L, ev, ws=0x1080) == S.STEM_ERR_WORKSPACE
    assert evict(L, ev, ws_bytes=255) == S.STEM_ERR_WORKSPACE


def test_oracle_eviction_rule_by_hand():
    w = np.array([0.0, 5.0, 1.0, np.nan, 5.0, 9.0, 0.5])
    assert O.evict_keep(w, 7, 7, 0, 0).tolist() == list(range(7))
    assert O.evict_keep(w, 7, 3, 0, 0).tolist() == [1, 4, 5]
    assert O.evict_keep(w, 7, 2, 0, 0).tolist() == [1, 5]             # the lower of two equal weights
    assert O.evict_keep(w, 7, 4, 1, 2).tolist() == [0, 1, 5, 6]       # sink, heaviest, recent
    assert O.evict_keep(w, 7, 6, 0, 0).tolist() == [0, 1, 2, 4, 5, 6]  # NaN goes first
