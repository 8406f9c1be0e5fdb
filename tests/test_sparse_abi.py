"""Host-only checks of the indexer's, the sparse and the tree attention's
entry points: each call breaks one rule, so none of them reaches a launch.
(Fake addresses, never dereferenced.)"""
import pytest
import torch

from paged_quantized_kv_gb300 import build as kbuild
from paged_quantized_kv_gb300 import kvq

A = 0x10000
SHAPE, NULL, ALIGN = kvq.KVQ_ERR_SHAPE, kvq.KVQ_ERR_NULL, kvq.KVQ_ERR_ALIGN
ARG, OK = kvq.KVQ_ERR_ARG, kvq.KVQ_OK


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq.lib()


ATTENTION = dict(query=A, query_stride0=1024, dtype=0, total_q=4, num_seqs=2,
                 cu_q_lens=A, max_q_len=4, num_q_heads=8, num_kv_heads=2,
                 head_size=128, key_cache=A, value_cache=A,
                 page_stride=2 * 2 * 16 * 72, block_size=16, num_blocks=8,
                 layout=0, block_table=A, block_table_stride=4,
                 max_blocks_per_seq=4, context_lens=A, max_context_len=0)
REST = dict(k_scale=A, v_scale=A, scale=0.1, workspace=A,
            workspace_bytes=1 << 40, out=A, out_stride0=1024, flags=0,
            dev_error=None, stream=None)
ATTENTION_BAD = [
    (dict(dtype=2), kvq.KVQ_ERR_DTYPE), (dict(layout=2), kvq.KVQ_ERR_LAYOUT),
    (dict(flags=4), ARG), (dict(flags=16), ARG), (dict(total_q=-1), SHAPE),
    (dict(total_q=(1 << 25) + 1), SHAPE), (dict(num_seqs=-1), SHAPE),
    (dict(num_seqs=(1 << 20) + 1), SHAPE), (dict(max_q_len=-1), SHAPE),
    (dict(max_context_len=-1), SHAPE), (dict(num_q_heads=7), SHAPE),
    (dict(head_size=64), SHAPE), (dict(block_size=6), SHAPE),
    (dict(block_table_stride=3), SHAPE),
    (dict(page_stride=16 * 2 * 72 - 16), SHAPE),
    (dict(query_stride0=1016), SHAPE), (dict(out_stride0=1016), SHAPE),
    (dict(scale=float("nan")), ARG), (dict(query=None), NULL),
    (dict(cu_q_lens=None), NULL), (dict(block_table=None), NULL),
    (dict(context_lens=None), NULL), (dict(workspace=None), NULL),
    (dict(out=None), NULL), (dict(query=A + 8), ALIGN),
    (dict(out_stride0=1028), ALIGN), (dict(key_cache=A + 8), ALIGN),
    (dict(workspace=A + 16), ALIGN),
    (dict(workspace_bytes=100), kvq.KVQ_ERR_SCRATCH),
    (dict(total_q=0, query=None, out=None), OK), (dict(num_seqs=0), OK),
]


def call(fn, first, kw, last):
    args = dict(ATTENTION, **first, **REST)
    args.update(kw)
    return fn(*args.values())


@pytest.mark.parametrize("kw,code", ATTENTION_BAD + [
    (dict(mask=None), NULL), (dict(mask=A + 2), ALIGN),
    (dict(words=0), SHAPE), (dict(words=33, mask_stride=33), SHAPE),
    (dict(mask_stride=1), SHAPE), (dict(total_q=0, mask=None), OK)])
def test_tree(lib, kw, code):
    assert call(lib.kvq_tree_attention_nvfp4,
                dict(mask=A, mask_stride=2, words=2), kw, None) == code


@pytest.mark.parametrize("kw,code", ATTENTION_BAD + [
    (dict(selected=None), NULL), (dict(selected=A + 2), ALIGN),
    (dict(top=0), SHAPE), (dict(top=-1), SHAPE), (dict(stride=7), SHAPE),
    (dict(sel=0), SHAPE), (dict(sel=24), SHAPE), (dict(sel=-16), SHAPE),
    (dict(sel=1 << 20, top=2, stride=2), SHAPE),
    (dict(total_q=0, selected=None), OK)])
def test_sparse(lib, kw, code):
    assert call(lib.kvq_sparse_attention_nvfp4,
                dict(selected=A, stride=8, top=8, sel=32), kw, None) == code


def test_sparse_workspace(lib):
    f = lib.kvq_sparse_attention_workspace_bytes
    one = f(1, 1, 8, 2, 8, 32, 16, 64)
    assert 0 < one <= f(5000, 4, 64, 8, 32, 64, 16, 4096)
    for bad in [(-1, 1, 8, 2, 8, 32, 16, 64), (1, -1, 8, 2, 8, 32, 16, 64),
                (1, 1, 0, 2, 8, 32, 16, 64), (1, 1, 7, 2, 8, 32, 16, 64),
                (1, 1, 8, 0, 8, 32, 16, 64), (1, 1, 8, 2, 0, 32, 16, 64),
                (1, 1, 8, 2, 8, 24, 16, 64), (1, 1, 8, 2, 8, 32, 0, 64),
                (1, 1, 8, 2, 8, 32, 16, -1), (1, 1, 17, 1, 8, 32, 16, 64),
                (1, 1, 1024, 1, 8, 32, 16, 64)]:
        assert f(*bad) == -1


@pytest.mark.parametrize("sel,top,blocks", [(64, 32, 2048), (16, 8, 512),
                                            (128, 4, 8192), (48, 8, 100)])
def test_sparse_workspace_does_not_shrink(lib, sel, top, blocks):
    """Neither with the rows nor with the sequences, also where its parts
    reach their limits."""
    f = lib.kvq_sparse_attention_workspace_bytes
    sizes = [0, 1, 4, 5, 64, 1000, 4096, 5000, 100000, 1 << 20, 1 << 25]
    for Hq, Hkv in [(8, 8), (64, 8), (16, 1)]:
        for n in [0, 1, 7, 1000, 65536]:
            at = [f(t, n, Hq, Hkv, top, sel, 16, blocks) for t in sizes]
            assert at == sorted(at) and at[0] > 0
        for t in sizes:
            at = [f(t, n, Hq, Hkv, top, sel, 16, blocks)
                  for n in [0, 1, 7, 1000, 30000, 65536]]
            assert at == sorted(at)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), kvq.KVQ_ERR_DTYPE), (dict(flags=4), ARG),
    (dict(scale=float("inf")), ARG), (dict(total_q=-1), SHAPE),
    (dict(total_q=(1 << 25) + 1), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=1025, q_stride=1025 * 64, w_stride=1025), SHAPE),
    (dict(D=48), SHAPE), (dict(D=512, q_stride=4096), SHAPE),
    (dict(q_stride=504), SHAPE), (dict(w_stride=7), SHAPE),
    (dict(q=None), NULL), (dict(weights=None), NULL),
    (dict(out=None), NULL), (dict(w_out=None), NULL),
    (dict(q=A + 8), ALIGN), (dict(q_stride=516), ALIGN),
    (dict(out=A + 8), ALIGN), (dict(weights=A + 2), ALIGN),
    (dict(w_out=A + 1), ALIGN), (dict(total_q=0, q=None), OK)])
def test_quantize(lib, kw, code):
    args = dict(q=A, q_stride=512, dtype=0, weights=A, w_stride=8, scale=1.0,
                total_q=4, heads=8, D=64, out=A, w_out=A, flags=0,
                stream=None)
    args.update(kw)
    assert lib.kvq_quantize_indexer_q(*args.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(flags=4), ARG), (dict(total_q=-1), SHAPE),
    (dict(total_q=(1 << 25) + 1), SHAPE), (dict(num_seqs=-1), SHAPE),
    (dict(num_seqs=(1 << 20) + 1), SHAPE), (dict(max_q=-1), SHAPE),
    (dict(heads=0), SHAPE),
    (dict(heads=129, q_stride=129 * 128, w_stride=129), SHAPE),
    (dict(D=48), SHAPE), (dict(D=256, q_stride=2048), SHAPE),
    (dict(block=0), SHAPE), (dict(num_blocks=-1), SHAPE),
    (dict(width=-1), SHAPE), (dict(bt_stride=3), SHAPE),
    (dict(sel=48), SHAPE), (dict(sel=256), SHAPE), (dict(sel=8), SHAPE),
    (dict(columns=-1), SHAPE), (dict(s_stride=7), SHAPE),
    (dict(columns=(1 << 20) + 1, s_stride=1 << 21), SHAPE),
    (dict(q_stride=1008), SHAPE), (dict(w_stride=7), SHAPE),
    (dict(block_stride=64 * 132 - 16), SHAPE),
    (dict(q=None), NULL), (dict(weights=None), NULL), (dict(cu=None), NULL),
    (dict(cache=None), NULL), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(scores=None), NULL),
    (dict(q=A + 8), ALIGN), (dict(q_stride=1032), ALIGN),
    (dict(weights=A + 2), ALIGN), (dict(cache=A + 8), ALIGN),
    (dict(block_stride=64 * 132 + 8), ALIGN), (dict(cu=A + 2), ALIGN),
    (dict(table=A + 1), ALIGN), (dict(lens=A + 2), ALIGN),
    (dict(scores=A + 2), ALIGN), (dict(total_q=0, q=None), OK),
    (dict(num_seqs=0), OK), (dict(columns=0), OK)])
def test_score(lib, kw, code):
    args = dict(q=A, q_stride=1024, weights=A, w_stride=8, total_q=4,
                num_seqs=2, cu=A, max_q=4, heads=8, D=128, cache=A,
                block_stride=64 * 132, num_blocks=8, block=64, table=A,
                bt_stride=4, width=4, lens=A, sel=64, scores=A, s_stride=8,
                columns=8, flags=0, err=None, stream=None)
    args.update(kw)
    assert lib.kvq_score_blocks_indexer_k(*args.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(flags=4), ARG), (dict(columns=-1), SHAPE),
    (dict(s_stride=7), SHAPE), (dict(total_q=-1), SHAPE),
    (dict(total_q=(1 << 25) + 1), SHAPE), (dict(num_seqs=-1), SHAPE),
    (dict(num_seqs=(1 << 20) + 1), SHAPE), (dict(sel=0), SHAPE),
    (dict(sel=1 << 24), SHAPE), (dict(top=0), SHAPE), (dict(stride=3), SHAPE),
    (dict(first=-1), ARG), (dict(last=-1), ARG),
    (dict(first=3, last=2), ARG), (dict(first=5), ARG),
    (dict(first=(1 << 31) - 1, last=(1 << 31) - 1), ARG),
    (dict(scores=None), NULL), (dict(cu=None), NULL), (dict(lens=None), NULL),
    (dict(selected=None), NULL), (dict(scores=A + 2), ALIGN),
    (dict(cu=A + 2), ALIGN), (dict(lens=A + 2), ALIGN),
    (dict(selected=A + 2), ALIGN), (dict(total_q=0, scores=None), OK),
    (dict(num_seqs=0), OK)])
def test_select(lib, kw, code):
    args = dict(scores=A, s_stride=8, columns=8, total_q=4, num_seqs=2, cu=A,
                lens=A, sel=64, first=1, last=2, selected=A, stride=4, top=4,
                flags=0, err=None, stream=None)
    args.update(kw)
    assert lib.kvq_select_blocks(*args.values()) == code


# ---------------------------------------------------------------------------
# the binding (host tensors: each call is refused before the library's)
# ---------------------------------------------------------------------------
def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def refused(code, fn, *args, **kw):
    with pytest.raises(kvq.KvqError) as e:
        fn(*args, **kw)
    assert e.value.status == code


def attention_args():
    kv, kc, vc = kvq.alloc_nvfp4_cache(4, 16, 2, 128, device="cpu")
    q = torch.zeros(5, 8, 128, dtype=torch.bfloat16)
    return [q, kc, vc, i32(2, 4), i32(3), i32(2)], [
        torch.ones(1), torch.ones(1), 0.1, torch.empty_like(q), 3]


def test_binding_tree(lib):
    a, z = attention_args()
    f = kvq.kvq_tree_attention_nvfp4
    refused(ARG, f, *a, i32(5, 1), *z)             # host memory
    refused(SHAPE, f, *a, i32(4, 1), *z)
    refused(SHAPE, f, *a, i32(5), *z)
    refused(SHAPE, f, *a, i32(2, 5).t(), *z)
    refused(kvq.KVQ_ERR_DTYPE, f, *a, i32(5, 1).long(), *z)


def test_binding_sparse(lib):
    a, z = attention_args()
    f = kvq.kvq_sparse_attention_nvfp4
    refused(ARG, f, *a, i32(5, 3), 32, *z)
    refused(SHAPE, f, *a, i32(4, 3), 32, *z)
    refused(SHAPE, f, *a, i32(3, 5).t(), 32, *z)
    refused(kvq.KVQ_ERR_DTYPE, f, *a, i32(5, 3).long(), 32, *z)
    refused(kvq.KVQ_ERR_DTYPE, f, a[0].float(), *a[1:], i32(5, 3), 32, *z)


def test_binding_indexer(lib):
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    q8 = torch.zeros(4, 8, 64, dtype=torch.uint8)
    w = torch.zeros(4, 8)
    f = kvq.kvq_quantize_indexer_q
    refused(ARG, f, q, w, 1.0, q8, w.clone())
    refused(SHAPE, f, q, w[:, :7], 1.0, q8, w)
    refused(SHAPE, f, q, w, 1.0, q8[:, :7], w)
    refused(SHAPE, f, q.transpose(0, 1), w, 1.0, q8.transpose(0, 1), w)
    refused(kvq.KVQ_ERR_DTYPE, f, q.float(), w, 1.0, q8, w)
    refused(kvq.KVQ_ERR_DTYPE, f, q, w.double(), 1.0, q8, w)
    refused(kvq.KVQ_ERR_DTYPE, f, q, w, 1.0, q8.int(), w)
    cache = torch.zeros(6, 16, 68, dtype=torch.uint8)
    s = torch.zeros(4, 5)
    f = kvq.kvq_score_blocks_indexer_k
    refused(ARG, f, q8, w, cache, i32(2, 3), i32(3), i32(2), s, 64, 2)
    refused(SHAPE, f, q8, w, cache, i32(2, 3), i32(2), i32(2), s, 64, 2)
    refused(SHAPE, f, q8, w, cache, i32(1, 3), i32(3), i32(2), s, 64, 2)
    refused(SHAPE, f, q8, w, cache[:, :, :60], i32(2, 3), i32(3), i32(2), s,
            64, 2)
    refused(SHAPE, f, q8, w, cache.view(6, -1), i32(2, 3), i32(3), i32(2), s,
            64, 2)
    refused(SHAPE, f, q8, w, cache.view(6, -1), i32(2, 3), i32(3), i32(2), s,
            64, 2, block_size=17)
    refused(SHAPE, f, q8, w, cache, i32(2, 3), i32(3), i32(2), s[:3], 64, 2)
    refused(kvq.KVQ_ERR_DTYPE, f, q8, w, cache, i32(2, 3), i32(3), i32(2),
            s.half(), 64, 2)
    f = kvq.kvq_select_blocks
    refused(ARG, f, s, i32(3), i32(2), i32(4, 2), 64)
    refused(SHAPE, f, s, i32(3), i32(2), i32(3, 2), 64)
    refused(SHAPE, f, s, i32(2), i32(2), i32(4, 2), 64)
    refused(kvq.KVQ_ERR_DTYPE, f, s, i32(3), i32(2), i32(4, 2).long(), 64)


@pytest.mark.parametrize("sel,top", [(16, 8), (64, 32), (128, 4)])
def test_sparse_workspace_does_not_shrink_with_the_table(lib, sel, top):
    """Also beyond the contexts that tiles can name: a call on a wide table
    whose longest context is shorter has them."""
    f = lib.kvq_sparse_attention_workspace_bytes
    edge = 8192 * sel // 16
    widths = [0, 1, 64, 2048, edge - 1, edge, edge + 1, 2 * edge, 1 << 22]
    for total, n in [(1, 1), (100, 3), (1024, 1), (5000, 70)]:
        at = [f(total, n, 64, 8, top, sel, 16, w) for w in widths]
        assert at == sorted(at)
        assert at[-1] == at[5]


def test_binding_dimensions(lib):
    """Tensors of fewer or more dimensions are refused as such."""
    a, z = attention_args()
    for bad in (torch.zeros((), dtype=torch.bfloat16),
                torch.zeros(5, dtype=torch.bfloat16), a[0][0], a[0][None]):
        refused(SHAPE, kvq.kvq_tree_attention_nvfp4, bad, *a[1:], i32(5, 1),
                *z)
        refused(SHAPE, kvq.kvq_sparse_attention_nvfp4, bad, *a[1:], i32(5, 3),
                32, *z)
        refused(SHAPE, kvq.sparse_attention_workspace, bad, i32(5, 3), a[1],
                a[3], 32)
    f = kvq.sparse_attention_workspace
    refused(SHAPE, f, a[0], i32(5), a[1], a[3], 32)
    refused(SHAPE, f, a[0], i32(5, 3), a[1][0], a[3], 32)
    refused(SHAPE, f, a[0], i32(5, 3), a[1], a[3][0], 32)
    s = torch.zeros(4, 5)
    for bad in (s[0], s[None], torch.zeros(())):
        refused(SHAPE, kvq.kvq_select_blocks, bad, i32(3), i32(2), i32(4, 2),
                64)
