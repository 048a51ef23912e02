"""Pages of the shared prefix that lie outside the cache: read as slot 0 and reported, by both
kernels that read prefixes; and pages that several sequences share."""
import pytest
import torch

from block_sparse_attention_oam_b200 import stem as S
from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("batch", [3, 40])       # decode_kernel's rows, and prefix_kernel's
def test_a_prefix_page_outside_the_cache(batch, dtype):
    s = D.Setup([5] * batch, Hq=8, Hkv=2, d=128, prefix=300, seed=70, dtype=dtype)
    for c in (s.cache.k_cache, s.cache.v_cache):     # slot 0 may be one that nobody uses (NaN)
        c.view(torch.uint8)[0] = c.view(torch.uint8)[int(s.prefix_table[0])]
    for at in (1, 4):                                # inside, and the last page, cut by the prefix's end
        table = s.prefix_table.clone()
        table[at] = 0
        want = s.call(prefix_table=table).clone()
        for bad in (-1, s.cache.k_cache.shape[0], 1 << 30):
            table[at] = bad
            ws = S.decode_workspace(s.dec)
            out = S.stem_decode(s.dec, s.q, s.cache, s.kv_lens, prefix_table=table, ws=ws)
            with pytest.raises(S.StemError) as e:
                S.query_status(ws)
            assert e.value.status == S.STEM_ERR_BOUNDS
            assert torch.equal(out, want)


def test_sequences_that_share_pages():
    """Two sequences over the same pages, the second shorter, are two sequences over copies."""
    s = D.Setup([700, 650], Hq=8, Hkv=2, d=128, seed=71, weights=True)
    s.cache.block_table[1] = s.cache.block_table[0]
    s.kv[1] = tuple(x[:650] for x in s.kv[0])
    s.check(s.call())
