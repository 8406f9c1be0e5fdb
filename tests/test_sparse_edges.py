"""kvq_sparse_attention_nvfp4 on the GPU where its tiles begin and end: block
tables much wider than the contexts, NaN scales in several blocks of a
tile."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.sparse_models import listed_tokens
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


def check_v_nan(c, b, sees, places, bits=0):
    """V scales (token, group) of sequence b made NaN: rows that see the token
    have NaN in the group's columns, all else is as without it."""
    plain = [a.copy() for a in c.ref()]
    n, L = int(c.cu[b + 1] - c.cu[b]), int(c.lens[b])
    nan = np.zeros((c.q.shape[0], 128), dtype=bool)
    for t, g in places:
        c.pages.set_scale(1, c.table[b, t // c.B], t % c.B, 0, g, 0x7F)
        for i in range(n):
            if sees(b, i, c.cu[b] + i, n, L)[t]:
                nan[c.cu[b] + i, 16 * g:16 * g + 16] = True
    got = c.run(bits=bits)
    full = np.broadcast_to(nan[:, None], got.shape)
    assert np.isnan(got[full]).all() and np.isfinite(got[~full]).all()
    got[full] = plain[0][full] = 0
    c.check(got, tuple(plain))
    return nan.any(1)


def listed_case(mixed):
    """Rows of four kinds in turn, which select both, one or the other or
    neither of blocks 6 and 8, the third and the fourth of their item's."""
    c = Sparse([64], [400], sel=16, top=9, hq=8, hkv=1)
    for r in range(64):
        e = [0, 3, 10, 12, 13, 16, 19]
        e += [6] if not mixed or r % 4 in (0, 2) else []
        e += [8] if not mixed or r % 4 in (0, 1) else []
        c.selected[r] = sorted(e) + [-1] * (9 - len(e))
    return c


# (8 heads to a KV head: items of 32 tokens; blocks 6 and 8 are in one quarter
# of their tile, 8 and 16 in two tiles)
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("places", [
    [(6 * 16 + 3, 0), (8 * 16, 0)], [(6 * 16, 5), (8 * 16 + 15, 5)],
    [(8 * 16 + 7, 2), (6 * 16 + 7, 2), (16 * 16 + 1, 2)],
    [(6 * 16 + 1, 1), (8 * 16 + 1, 7), (19 * 16 + 9, 1)]])
def test_nan_in_blocks_of_one_tile(tiles_library, telling_library,
                                   monkeypatch, mixed, places):
    """Rows that see the second block with a NaN scale and not the first."""
    c = listed_case(mixed)
    use(monkeypatch, tiles_library)
    hit = check_v_nan(c, 0, listed_tokens(c.selected, 16), places)
    assert hit.any() and hit.all() != (mixed and len(places) == 2)
    use(monkeypatch, telling_library)
    c.upload()
    c.call()
    torch.cuda.synchronize()
    assert int(c.err.item()) == kvq.KVQ_DEVERR_TIMEOUT   # (it has tiles)


@pytest.mark.parametrize("at", [0, 1, 14, 15])
def test_nan_behind_a_row_in_its_own_block(tiles_library, monkeypatch, at):
    """The block in which rows lie, listed by all: rows before the token do
    not see it, those from it on do."""
    c = Sparse([64], [400], sel=16, top=9, hq=8, hkv=1)
    for r in range(64):
        own = (336 + r) // 16
        e = sorted({0, 3, 6, 8, 10, 12, 13, own})
        c.selected[r] = e + [-1] * (9 - len(e))
    use(monkeypatch, tiles_library)
    places = [(16 * e + at, 4) for e in (21, 22, 24)]
    hit = check_v_nan(c, 0, listed_tokens(c.selected, 16), places)
    assert hit.any() and not hit.all() or at == 0
