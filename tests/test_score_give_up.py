"""Block scores whose wait gives up end soon.  In a test-only build an epilogue
warp of every other thread block gives up at once, without a wait that runs
out; what is left is to see the copies and the products in flight through,
which takes microseconds.  No warp may wait for a copy that nobody has begun:
that would take the limit of a wait once more, and again for each of them."""
import time

import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.test_indexer_selection import Scores
from tests.variant_build import build_variant

pytestmark = pytest.mark.gpu

LIMIT = 0.4  # seconds


@pytest.fixture(scope="module")
def giving_up(tmp_path_factory):
    return build_variant(tmp_path_factory.mktemp("kvq_soon"), {
        "score_blocks.cu": {"KVQ_TEST_SCORE_GIVE_UP": 1,
                            "KVQ_WAIT_LIMIT_NS": int(LIMIT * 1e9)}})


# (more tiles a thread block than it has stages, so that the warps that copy
# wait for an empty one; forms of one and of two such warps)
@pytest.mark.parametrize("q_lens,lens", [
    ([1] * 40, [9000] * 40), ([2] * 30, [12000] * 30), ([64], [40000]),
    ([7] * 40, [9000] * 40)])
def test_gives_up_within_the_limit(giving_up, monkeypatch, q_lens, lens):
    c = Scores(q_lens, lens, heads=32, seed=len(q_lens))
    want = c.run()
    monkeypatch.setattr(kvq, "LIB_PATH", giving_up)
    monkeypatch.setattr(kvq, "_lib", None)
    c.run(bits=kvq.KVQ_DEVERR_TIMEOUT)  # (loads the kernel)
    torch.cuda.synchronize()
    since = time.perf_counter()
    got = c.run(bits=kvq.KVQ_DEVERR_TIMEOUT)
    assert time.perf_counter() - since < LIMIT
    left = got == 77.0
    assert left.any() and (got[~left] == want[~left]).all()
    assert np.isfinite(want).any()
