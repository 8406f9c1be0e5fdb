"""kvq_tree_attention_nvfp4 on the GPU: chunks longer than max_q_len, and NaN
scales of several drafts, by rows and by tiles."""
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.sparse_models import tree_tokens
from tests.test_sparse_edges import check_v_nan
from tests.test_tree_attention import Tree
from tests.variant_build import build_variant

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens", [[20, 1, 4], [70, 1, 9], [2, 0, 5, 1, 3]])
@pytest.mark.parametrize("max_q", [0, 1, 2, 3])
def test_trees_beyond_max_q_len(max_q, q_lens):
    """Flagged, their rows left as they were, and the others right."""
    c = Tree(q_lens, [n + 61 * n for n in q_lens], hq=8, hkv=2, seed=max_q)
    got, ref = c.run(bits=kvq.KVQ_DEVERR_SEQ, max_q=max_q), c.ref()
    for b, n in enumerate(q_lens):
        rows = slice(c.cu[b], c.cu[b + 1])
        if n > max(max_q, 1):
            assert (got[rows] == 77.0).all()
            got[rows] = ref[0][rows]
    c.check(got, ref)


@pytest.mark.parametrize("max_q", [20, 500, 1 << 30])
def test_max_q_len_beyond_the_trees(max_q):
    c = Tree([20, 1, 4], [500, 300, 64], hq=8, hkv=2)
    c.check(c.run(max_q=max_q))


# contexts after which the drafts lie in one quarter of a tile, in two, in two
# tiles, and behind many thread blocks' shares
@pytest.mark.parametrize("ctx", [0, 100, 118, 121, 9000])
@pytest.mark.parametrize("n", [12, 20, 70])
def test_nan_of_two_drafts_by_tiles(n, ctx):
    """Rows of trees that go by tiles and see the second draft with a NaN
    scale and not the first, the first and not the second, both, neither."""
    c = Tree([n, n], [300, n + ctx], hq=2, hkv=1, seed=n + ctx)
    j0, j1 = n - 8, n - 6
    for i in range(n):
        r = n + i
        c.mask[r] = 0
        for j in [i] + ([j0] if i % 4 in (0, 2) else []) + (
                [j1] if i % 4 in (0, 1) else []):
            c.mask[r, j // 32] |= 1 << j % 32
    c.mask[n + j0] = c.mask[n + 3]      # (neither, nor itself)
    hit = check_v_nan(c, 1, tree_tokens(c.mask),
                      [(ctx + j0, 0), (ctx + j1, 0), (ctx + j1, 6)])
    assert hit.any() and not hit[n:].all() and not hit[:n].any()


@pytest.mark.parametrize("ctx", [0, 30, 100, 125])
@pytest.mark.parametrize("n", [3, 8])
def test_nan_of_two_drafts_by_rows(n, ctx):
    c = Tree([n], [n + ctx], hq=2, hkv=1)
    c.mask[:, 0] = [1 << i for i in range(n)]
    c.mask[2, 0] |= 0b10
    hit = check_v_nan(c, 0, tree_tokens(c.mask), [(ctx, 0), (ctx + 1, 0)])
    assert hit[:3].all() and not hit[3:].any()


# ---------------------------------------------------------------------------
# by rows or by tiles
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def telling_library(tmp_path_factory):
    """A softmax warp of the tiles' kernel gives up: a call says
    KVQ_DEVERR_TIMEOUT if it has tiles."""
    return build_variant(tmp_path_factory.mktemp("kvq_tell"), {
        "chunk_attention.cu": {"KVQ_TEST_GIVE_UP": 1,
                               "KVQ_WAIT_LIMIT_NS": 20000000}})


# per: tokens of the contexts for each multiprocessor and KV head.  Measured
# well away from where both are even: 8 drafts at 2300 took 73 to 79 us by rows
# and 52 to 63 by tiles, at 600 24 to 28 and 27 to 38.
@pytest.mark.parametrize("drafts,per,G,tiles", [
    (4, 6000, 8, False), (5, 2300, 8, False), (5, 6000, 8, True),
    (6, 1500, 8, False), (6, 4000, 8, True), (7, 1000, 8, False),
    (7, 2300, 8, True), (8, 600, 8, False), (8, 2300, 8, True),
    (8, 600, 1, False), (8, 2300, 1, True), (5, 600, 16, False),
    (5, 2300, 16, True), (8, 300, 16, False), (8, 1000, 16, True),
    (9, 100, 8, True)])
def test_rows_or_tiles(telling_library, monkeypatch, drafts, per, G, tiles):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = Tree([drafts] * 4, [per * sms // 8] * 4, hq=2 * G, hkv=2)
    monkeypatch.setattr(kvq, "LIB_PATH", telling_library)
    monkeypatch.setattr(kvq, "_lib", None)
    c.upload()
    c.call(max_context_len=per * sms // 8)
    torch.cuda.synchronize()
    assert int(c.err.item()) == (kvq.KVQ_DEVERR_TIMEOUT if tiles else 0)
