"""Host-only checks of the chunk attention's and the page operators' entry
points: each call breaks one rule, so none of them reaches a launch.  (Fake
addresses, never dereferenced.)"""
import ctypes

import pytest
import torch

from paged_quantized_kv_gb300 import build as kbuild
from paged_quantized_kv_gb300 import kvq

A = 0x10000
SHAPE, NULL, ALIGN = kvq.KVQ_ERR_SHAPE, kvq.KVQ_ERR_NULL, kvq.KVQ_ERR_ALIGN


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq.lib()


def chunk(lib, **kw):
    args = dict(query=A, query_stride0=1024, dtype=0, total_q=4, num_seqs=2,
                cu_q_lens=A, max_q_len=4, num_q_heads=8, num_kv_heads=2,
                head_size=128, key_cache=A, value_cache=A,
                page_stride=2 * 2 * 16 * 72, block_size=16, num_blocks=8,
                layout=0, block_table=A, block_table_stride=4,
                max_blocks_per_seq=4, context_lens=A, max_context_len=0,
                k_scale=A, v_scale=A, scale=0.1, workspace=A,
                workspace_bytes=1 << 40, out=A, out_stride0=1024, flags=0,
                dev_error=None, stream=None)
    args.update(kw)
    return lib.kvq_chunk_attention_nvfp4(*args.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), kvq.KVQ_ERR_DTYPE),
    (dict(layout=2), kvq.KVQ_ERR_LAYOUT),
    (dict(flags=4), kvq.KVQ_ERR_ARG),
    (dict(flags=16), kvq.KVQ_ERR_ARG),
    (dict(total_q=-1), SHAPE), (dict(total_q=(1 << 25) + 1), SHAPE),
    (dict(num_seqs=-1), SHAPE), (dict(num_seqs=(1 << 20) + 1), SHAPE),
    (dict(max_q_len=-1), SHAPE), (dict(max_context_len=-1), SHAPE),
    (dict(num_q_heads=0), SHAPE), (dict(num_q_heads=7), SHAPE),
    (dict(num_q_heads=34, query_stride0=34 * 128, out_stride0=34 * 128),
     SHAPE),
    (dict(num_q_heads=1040, num_kv_heads=65, query_stride0=1040 * 128,
          out_stride0=1040 * 128, page_stride=65 * 16 * 72 * 2), SHAPE),
    (dict(head_size=64), SHAPE), (dict(block_size=6), SHAPE),
    (dict(block_size=0), SHAPE), (dict(num_blocks=-1), SHAPE),
    (dict(max_blocks_per_seq=-1), SHAPE),
    (dict(block_table_stride=3), SHAPE),
    (dict(page_stride=16 * 2 * 72 - 16), SHAPE),
    (dict(query_stride0=1016), SHAPE), (dict(out_stride0=1016), SHAPE),
    (dict(scale=float("nan")), kvq.KVQ_ERR_ARG),
    (dict(scale=float("inf")), kvq.KVQ_ERR_ARG),
    (dict(query=None), NULL), (dict(cu_q_lens=None), NULL),
    (dict(key_cache=None), NULL), (dict(value_cache=None), NULL),
    (dict(block_table=None), NULL), (dict(context_lens=None), NULL),
    (dict(k_scale=None), NULL), (dict(v_scale=None), NULL),
    (dict(workspace=None), NULL), (dict(out=None), NULL),
    (dict(query=A + 8), ALIGN), (dict(out=A + 8), ALIGN),
    (dict(query_stride0=1028), ALIGN), (dict(out_stride0=1028), ALIGN),
    (dict(key_cache=A + 8), ALIGN), (dict(value_cache=A + 4), ALIGN),
    (dict(page_stride=2 * 2 * 16 * 72 + 8), ALIGN),
    (dict(block_table=A + 2), ALIGN), (dict(cu_q_lens=A + 1), ALIGN),
    (dict(context_lens=A + 2), ALIGN), (dict(workspace=A + 16), ALIGN),
    (dict(workspace_bytes=100), kvq.KVQ_ERR_SCRATCH),
    (dict(total_q=0, query=None, out=None), kvq.KVQ_OK),
    (dict(num_seqs=0), kvq.KVQ_OK),
])
def test_chunk_attention(lib, kw, code):
    assert chunk(lib, **kw) == code


POOL = dict(ref_count=A, num_blocks=100, block_table=A, block_table_stride=8,
            num_rows=6, max_blocks_per_seq=8, seq_lens=A)
POOL_BAD = [
    (dict(num_blocks=-1), SHAPE), (dict(num_blocks=(1 << 31) - 1), SHAPE),
    (dict(num_rows=-1), SHAPE), (dict(num_rows=(1 << 18) + 1), SHAPE),
    (dict(max_blocks_per_seq=-1), SHAPE),
    (dict(block_table_stride=7), SHAPE),
    (dict(ref_count=None), NULL), (dict(block_table=None), NULL),
    (dict(seq_lens=None), NULL), (dict(ref_count=A + 2), ALIGN),
    (dict(block_table=A + 1), ALIGN), (dict(seq_lens=A + 3), ALIGN),
    (dict(flags=4), kvq.KVQ_ERR_ARG), (dict(n=-1), SHAPE),
    (dict(n=4097), SHAPE), (dict(n=0), kvq.KVQ_OK),
    (dict(n=0, ref_count=None, ids=None), kvq.KVQ_OK),
    (dict(ids=None), NULL), (dict(ids=A + 2), ALIGN),
]
BLOCK_BAD = [(dict(block_size=0), SHAPE), (dict(block_size=-4), SHAPE),
             (dict(block_size=1 << 28), SHAPE)]


def call(fn, defaults, kw):
    args = dict(defaults)
    args.update(kw)
    return fn(*args.values())


@pytest.mark.parametrize("kw,code", POOL_BAD + BLOCK_BAD + [
    (dict(cu=None), NULL), (dict(slots=None), NULL), (dict(cu=A + 1), ALIGN),
    (dict(slots=A + 4), ALIGN), (dict(total=-1), SHAPE),
    (dict(total=1 << 31), SHAPE)])
def test_extend(lib, kw, code):
    assert call(lib.kvq_extend_sequences, dict(
        POOL, block_size=16, ids=A, cu=A, n=2, slots=A, total=9, flags=0,
        dev_error=None, stream=None), kw) == code


@pytest.mark.parametrize("kw,code", POOL_BAD + BLOCK_BAD + [
    (dict(children=None), NULL), (dict(src=None), NULL),
    (dict(dst=None), NULL), (dict(children=A + 2), ALIGN),
    (dict(src=A + 1), ALIGN), (dict(dst=A + 2), ALIGN),
    (dict(n=4096, block_size=1, max_blocks_per_seq=1 << 20,
          block_table_stride=1 << 20), SHAPE)])
def test_fork(lib, kw, code):
    assert call(lib.kvq_fork_sequences, dict(
        POOL, block_size=16, ids=A, children=A, n=2, src=A, dst=A, flags=0,
        dev_error=None, stream=None), kw) == code


@pytest.mark.parametrize("kw,code", POOL_BAD + BLOCK_BAD + [
    (dict(cu=None), NULL), (dict(keep=None), NULL), (dict(src=None), NULL),
    (dict(dst=None), NULL), (dict(cu=A + 1), ALIGN),
    (dict(keep=A + 2), ALIGN), (dict(src=A + 4), ALIGN),
    (dict(dst=A + 4), ALIGN), (dict(total=-1), SHAPE),
    (dict(total=1 << 31), SHAPE)])
def test_compact(lib, kw, code):
    assert call(lib.kvq_compact_sequences, dict(
        POOL, block_size=16, ids=A, keep=A, cu=A, n=2, src=A, dst=A, total=9,
        flags=0, dev_error=None, stream=None), kw) == code


@pytest.mark.parametrize("kw,code", POOL_BAD)
def test_free(lib, kw, code):
    assert call(lib.kvq_free_sequences, dict(
        POOL, ids=A, n=2, flags=0, dev_error=None, stream=None), kw) == code


def ptrs(*addresses):
    return (ctypes.c_void_p * len(addresses))(*addresses)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=1), kvq.KVQ_ERR_ARG), (dict(n=-1), SHAPE),
    (dict(pairs=-1), SHAPE), (dict(num_blocks=-1), SHAPE),
    (dict(page_bytes=0), SHAPE), (dict(page_stride=560), SHAPE),
    (dict(caches=None), NULL), (dict(caches=ptrs(A, 0)), NULL),
    (dict(src=None), NULL), (dict(dst=None), NULL),
    (dict(caches=ptrs(A, A + 8)), ALIGN), (dict(src=A + 2), ALIGN),
    (dict(dst=A + 2), ALIGN), (dict(page_stride=584), ALIGN),
    (dict(page_bytes=568), ALIGN),
    (dict(pairs=1 << 30, page_bytes=1 << 20, page_stride=1 << 20), SHAPE),
    (dict(pairs=1 << 17, page_bytes=1 << 58, page_stride=1 << 58), SHAPE),
    (dict(n=0, caches=None), kvq.KVQ_OK),
    (dict(pairs=0, src=None), kvq.KVQ_OK)])
def test_copy_pages(lib, kw, code):
    assert call(lib.kvq_copy_pages, dict(
        caches=ptrs(A, A), n=2, page_stride=576, page_bytes=576,
        num_blocks=10, src=A, dst=A, pairs=3, flags=0, dev_error=None,
        stream=None), kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(layout=2), kvq.KVQ_ERR_LAYOUT), (dict(flags=4), kvq.KVQ_ERR_ARG),
    (dict(n=-1), SHAPE), (dict(lists=-1), SHAPE), (dict(total=-1), SHAPE),
    (dict(total=1 << 31), SHAPE), (dict(num_blocks=-1), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE),
    (dict(head_size=96), SHAPE), (dict(head_size=8256), SHAPE),
    (dict(block_size=6), SHAPE), (dict(value_offset=2 * 16 * 72 - 16), SHAPE),
    (dict(page_stride=2 * 16 * 72 - 16), SHAPE),
    (dict(caches=None), NULL), (dict(caches=ptrs(0)), NULL),
    (dict(src=None), NULL), (dict(dst=None), NULL), (dict(cu=None), NULL),
    (dict(caches=ptrs(A + 4)), ALIGN), (dict(src=A + 4), ALIGN),
    (dict(dst=A + 4), ALIGN), (dict(cu=A + 2), ALIGN),
    (dict(value_offset=2 * 16 * 72 + 8), ALIGN),
    (dict(n=0), kvq.KVQ_OK), (dict(lists=0), kvq.KVQ_OK),
    (dict(total=0), kvq.KVQ_OK)])
def test_move_tokens(lib, kw, code):
    assert call(lib.kvq_move_tokens_nvfp4, dict(
        caches=ptrs(A), n=1, value_offset=2 * 16 * 72,
        page_stride=2 * 2 * 16 * 72, num_blocks=10, block_size=16, layout=0,
        heads=2, head_size=128, src=A, dst=A, total=5, cu=A, lists=1,
        flags=0, dev_error=None, stream=None), kw) == code


# ---------------------------------------------------------------------------
# the binding: host tensors, wrong types and shapes raise before a call
# ---------------------------------------------------------------------------
def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def i64(*shape):
    return torch.zeros(shape, dtype=torch.int64)


def refused(fn, code, *args, **kw):
    with pytest.raises(kvq.KvqError) as e:
        fn(*args, **kw)
    assert e.value.status == code


def chunk_args():
    kv, kc, vc = kvq.alloc_nvfp4_cache(4, 16, 2, 128, device="cpu", fill=0)
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    s = torch.ones(1)
    return dict(query=q, key_cache=kc, value_cache=vc, block_table=i32(2, 3),
                cu_q_lens=i32(3), context_lens=i32(2), k_scale=s, v_scale=s,
                scale=0.1, out=torch.zeros_like(q), max_q_len=3)


@pytest.mark.parametrize("kw,code", [
    (dict(), kvq.KVQ_ERR_ARG),                       # host tensors
    (dict(query=torch.zeros(3, 4, 128)), kvq.KVQ_ERR_DTYPE),
    (dict(out=torch.zeros(3, 4, 128, dtype=torch.float16)),
     kvq.KVQ_ERR_DTYPE),
    (dict(out=torch.zeros(2, 4, 128, dtype=torch.bfloat16)), SHAPE),
    (dict(query=torch.zeros(3, 4, 256, dtype=torch.bfloat16)[..., ::2]),
     SHAPE),
    (dict(cu_q_lens=i32(2)), SHAPE), (dict(cu_q_lens=i64(3)),
                                      kvq.KVQ_ERR_DTYPE),
    (dict(context_lens=i64(2)), kvq.KVQ_ERR_DTYPE),
    (dict(block_table=i64(2, 3)), kvq.KVQ_ERR_DTYPE),
    (dict(block_table=i32(1, 3)), SHAPE),
    (dict(block_table=i32(2, 6)[:, ::2]), SHAPE),
    (dict(k_scale=torch.ones(1, dtype=torch.float64)), kvq.KVQ_ERR_DTYPE),
    (dict(key_cache=torch.zeros(4, 16, 2, 72)), kvq.KVQ_ERR_DTYPE),
    (dict(key_cache=torch.zeros(4, 16, 2, 72, dtype=torch.uint8)), SHAPE),
    (dict(dev_error=i64(1)), kvq.KVQ_ERR_DTYPE),
])
def test_binding_chunk(lib, kw, code):
    args = chunk_args()
    args.update(kw)
    refused(kvq.kvq_chunk_attention_nvfp4, code, **args)


def test_binding_pool(lib):
    ref, table, lens = kvq.alloc_page_pool(8, 3, 4, device="cpu")
    ids = i32(2)
    for args, code in [
        ((ref, table, lens, ids, i32(3), i64(5), 4), kvq.KVQ_ERR_ARG),
        ((ref, table, lens, ids, i32(2), i64(5), 4), SHAPE),
        ((ref, table, lens, i64(2), i32(3), i64(5), 4), kvq.KVQ_ERR_DTYPE),
        ((ref, table, lens, ids, i32(3), i32(5), 4), kvq.KVQ_ERR_DTYPE),
        ((ref, table, lens[:2], ids, i32(3), i64(5), 4), SHAPE),
        ((ref, i32(1, 4).expand(3, 4), lens, ids, i32(3), i64(5), 4), SHAPE),
        ((ref, i32(3, 8)[:, ::2], lens, ids, i32(3), i64(5), 4), SHAPE),
        ((ref.long(), table, lens, ids, i32(3), i64(5), 4),
         kvq.KVQ_ERR_DTYPE),
        ((ref, table, lens, i32(4)[::2], i32(3), i64(5), 4), SHAPE),
    ]:
        refused(kvq.kvq_extend_sequences, code, *args)
    refused(kvq.kvq_fork_sequences, kvq.KVQ_ERR_ARG, ref, table, lens, ids,
            ids, i32(2), i32(2), 4)
    refused(kvq.kvq_fork_sequences, SHAPE, ref, table, lens, ids, i32(3),
            i32(2), i32(2), 4)
    refused(kvq.kvq_compact_sequences, kvq.KVQ_ERR_ARG, ref, table, lens,
            ids, i32(5), i32(3), i64(5), i64(5), 4)
    refused(kvq.kvq_compact_sequences, SHAPE, ref, table, lens, ids, i32(5),
            i32(3), i64(4), i64(5), 4)
    refused(kvq.kvq_free_sequences, kvq.KVQ_ERR_ARG, ref, table, lens, ids)
    refused(kvq.kvq_free_sequences, kvq.KVQ_ERR_DTYPE, ref, table, lens,
            i64(2))


def test_binding_moves(lib):
    c = torch.zeros(2, 6, 64, dtype=torch.uint8)
    for args, code in [
        ((c, i32(2), i32(2)), kvq.KVQ_ERR_ARG),
        ((list(c), i32(2), i32(2)), kvq.KVQ_ERR_ARG),
        ((c, i32(2), i32(3)), SHAPE), ((c, i64(2), i32(2)),
                                       kvq.KVQ_ERR_DTYPE),
        ((c.float(), i32(2), i32(2)), kvq.KVQ_ERR_DTYPE),
        (([], i32(2), i32(2)), SHAPE), ((c[0], i32(2), i32(2)), SHAPE),
        (([c[0], c[1, :3]], i32(2), i32(2)), SHAPE),
        (([c[0, :, ::2]], i32(2), i32(2)), SHAPE),
        ((c[:1].expand(2, 6, 64), i32(2), i32(2)), SHAPE),
    ]:
        refused(kvq.kvq_copy_pages, code, *args)
    kv, _, _ = kvq.alloc_nvfp4_cache(3, 4, 2, 64, device="cpu", fill=0)
    for args, kw, code in [
        (([kv], i64(3), i64(3), i32(2)), {}, kvq.KVQ_ERR_ARG),
        (([kv], i64(3), i64(2), i32(2)), {}, SHAPE),
        (([kv], i32(3), i64(3), i32(2)), {}, kvq.KVQ_ERR_DTYPE),
        (([kv], i64(3), i64(3), i64(2)), {}, kvq.KVQ_ERR_DTYPE),
        (([kv], i64(3), i64(3), i32(2)), dict(layout=3), kvq.KVQ_ERR_LAYOUT),
        (([kv, kv], i64(3), i64(3), i32(2)), {}, SHAPE),
        (([kv[:, 0]], i64(3), i64(3), i32(2)), {}, SHAPE),
        (([kv[..., :32]], i64(3), i64(3), i32(2)), {}, SHAPE),
    ]:
        refused(kvq.kvq_move_tokens_nvfp4, code, *args, **kw)


def test_workspace_and_status_strings(lib):
    assert lib.kvq_chunk_attention_workspace_bytes() > 0
    for bit in (kvq.KVQ_DEVERR_REF, kvq.KVQ_DEVERR_FULL):
        assert bit & (bit - 1) == 0
