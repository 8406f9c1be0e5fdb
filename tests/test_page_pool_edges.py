"""The page pool's calls at their edges: calls from two host threads, pages
that nobody holds, lists without entries, entries that need no page, table
entries that are no pages."""
import threading

import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.test_page_pool import dev

pytestmark = pytest.mark.gpu


def test_two_threads_with_pools_of_different_sizes():
    """Two host threads, each with a pool, a stream and a list of its own,
    whose kernels need different amounts of shared memory: no call of one is
    refused because of the other's.  (Calls of the C entries, made as fast as
    the threads can.)"""
    start, refused, states = threading.Barrier(2), [], {}

    def loop(name, rows, calls=20000):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ref, table, lens = kvq.alloc_page_pool(8, rows, 1)
            err, ids, cu = dev([0]), dev([rows - 1, 0]), dev([0, 3, 5])
            slots = torch.zeros(5, dtype=torch.int64, device="cuda")
            stream.synchronize()
            state = (ref.data_ptr(), 8, table.data_ptr(), 1, rows, 1,
                     lens.data_ptr())
            extend = state + (4, ids.data_ptr(), cu.data_ptr(), 2,
                              slots.data_ptr(), 5, 0, err.data_ptr(),
                              stream.cuda_stream)
            free = state + (ids.data_ptr(), 2, 0, err.data_ptr(),
                            stream.cuda_stream)
            L = kvq.lib()
            start.wait()
            for _ in range(calls):
                codes = (L.kvq_extend_sequences(*extend),
                         L.kvq_free_sequences(*free))
                if codes != (0, 0):
                    refused.append((name, codes))
                    break
            stream.synchronize()
            states[name] = (int(err.item()), int(ref.abs().sum().item()),
                            slots.tolist())

    threads = [threading.Thread(target=loop, args=a)
               for a in (("small", 170000), ("large", 1 << 18))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == []
    for state in states.values():
        assert state == (0, 0, [0, 1, 2, 4, 5])
