"""kvq_sparse_attention_nvfp4 on the GPU where its tiles begin and end: block
tables much wider than the contexts, NaN scales in several blocks of a
tile."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.test_sparse_attention import Sparse
from tests.variant_build import build_variant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tiles_library(tmp_path_factory):
    """Asks whether tiles pay however small the batch is."""
    return build_variant(tmp_path_factory.mktemp("kvq_tiles"), {
        "sparse_attention.cu": {"KVQ_SPARSE_ITEMS_FROM": 0}})


@pytest.fixture(scope="module")
def telling_library(tmp_path_factory):
    """The same, and a softmax warp of the tiles' kernel gives up: a call says
    KVQ_DEVERR_TIMEOUT if it has tiles."""
    return build_variant(tmp_path_factory.mktemp("kvq_tell"), {
        "sparse_attention.cu": {"KVQ_SPARSE_ITEMS_FROM": 0},
        "chunk_attention.cu": {"KVQ_TEST_GIVE_UP": 1,
                               "KVQ_WAIT_LIMIT_NS": 20000000}})


def use(monkeypatch, library):
    monkeypatch.setattr(kvq, "LIB_PATH", library)
    monkeypatch.setattr(kvq, "_lib", None)


def wide_case(pages):
    """64 rows that agree, with a block table of `pages` entries a row."""
    c = Sparse([64, 1], [900, 333], sel=16, top=9, near=1.0, hq=8, hkv=1)
    table = np.full((2, pages), -1, dtype=np.int32)
    table[:, :c.table.shape[1]] = c.table
    c.table = table
    return c


# 8192 blocks of 16 tokens are the most that tiles can name
@pytest.mark.parametrize("pages,longest,tiles", [
    (100, 0, True), (8192, 0, True), (8193, 0, False), (8193, 1000, True),
    (100000, 900, True), (100000, 16 * 8192, True),
    (100000, 16 * 8192 + 1, False), (100000, 0, False)])
def test_table_wider_than_the_contexts(tiles_library, telling_library,
                                       monkeypatch, pages, longest, tiles):
    c = wide_case(pages)
    use(monkeypatch, tiles_library)
    c.check(c.run(max_context_len=longest))
    use(monkeypatch, telling_library)
    c.upload()
    c.call(max_context_len=longest)
    torch.cuda.synchronize()
    assert int(c.err.item()) == (kvq.KVQ_DEVERR_TIMEOUT if tiles else 0)


def test_workspace_of_the_longest_context(tiles_library, monkeypatch):
    """A workspace for fewer pages than the table has, as many as
    max_context_len needs, is enough, and not one for fewer."""
    use(monkeypatch, tiles_library)
    c = wide_case(100000).upload()
    selected = torch.from_numpy(c.selected).cuda()
    for longest, needs in ((900, 900), (900, 4000), (0, 0)):
        ws = kvq.sparse_attention_workspace(c.qd, selected, c.kc, c.bt, c.sel,
                                            max_context_len=needs)
        c.check(c.run(max_context_len=longest, workspace=ws))
    small = kvq.sparse_attention_workspace(c.qd, selected, c.kc, c.bt, c.sel,
                                           max_context_len=100)
    with pytest.raises(kvq.KvqError) as e:
        c.run(max_context_len=900, workspace=small)
    assert e.value.status == kvq.KVQ_ERR_SCRATCH
