"""The problems of the decoding operators as objects: their numbers are those of the call."""
import dataclasses

import pytest

from block_sparse_attention_oam_b200 import build as B
from block_sparse_attention_oam_b200 import stem as S

GOOD = dict(num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=128, max_kv_len=1000)
PROBLEMS = [S.Decode(3, 8, 2, 128, max_kv_len=1000, dtype="fp8_e4m3", q_scale=0.5), S.Evict(3, 2, 128, max_kv_len=1000, budget=64)]


@pytest.mark.parametrize("p", PROBLEMS, ids=lambda p: type(p).__name__)
def test_a_problem_is_not_changed_behind_the_calls_back(p):
    for f in dataclasses.fields(p):
        with pytest.raises(dataclasses.FrozenInstanceError):
            setattr(p, f.name, getattr(p, f.name))


def test_another_problem_carries_its_own_numbers():
    a = PROBLEMS[0]
    b = dataclasses.replace(a, q_scale=0.25, q_len=4)
    assert (a._c.q_scale, a._c.q_len) == (0.5, 1) and (b._c.q_scale, b._c.q_len) == (0.25, 4)
    assert (b._c.num_seqs, b._c.max_kv_len, b._c.dtype) == (3, 1000, S.DT_FP8)
    c = dataclasses.replace(PROBLEMS[1], budget=32, recent=8)
    assert (c._c.budget, c._c.recent, c._c.max_kv_len) == (32, 8, 1000)


@pytest.mark.parametrize("kw", [dict(q_scale=1e30, k_scale=1e30), dict(q_scale=3e38, k_scale=20.0),
                                dict(q_scale=1e20, k_scale=1e10, softmax_scale=1e10)])
def test_scores_scaled_beyond_float32_are_refused(kw):
    """Each factor is finite, their product is not: 0 times it would be NaN."""
    B.build()
    with pytest.raises(S.StemError, match="beyond float32"):
        S.Decode(**GOOD, dtype="fp8_e4m3", **kw).workspace_bytes()
    if "softmax_scale" not in kw:        # the same factors, another sigma
        assert S.Decode(**GOOD, dtype="fp8_e4m3", softmax_scale=1e-30, **kw).workspace_bytes() > 0


def test_a_sigma_beyond_float32_is_refused():
    with pytest.raises(S.StemError, match="beyond float32"):
        S.Decode(**GOOD, softmax_scale=3e38).workspace_bytes()
    assert S.Decode(**GOOD, softmax_scale=2e38).workspace_bytes() > 0
    assert S.Decode(**GOOD, q_scale=1e30, k_scale=1e30).workspace_bytes() > 0      # BF16 has no scales
