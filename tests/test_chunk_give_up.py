"""Failure detection of the chunk attention without a GPU fault.  In a
test-only build one softmax warp of most thread blocks gives up at the end of
its first or second segment, as if its bounded wait had run out.  The call
must end, report KVQ_DEVERR_TIMEOUT, leave the rows that are concerned as they
were (whole heads' rows, those joined from several thread blocks too) and
write the others right; the regular library works afterwards."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import build as kbuild
from paged_quantized_kv_gb300 import kvq
from tests.test_chunk_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def giving_up(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("kvq_give_up") / "libkvq_give_up.so")
    kbuild.build(defines={"KVQ_TEST_GIVE_UP": 1,
                          "KVQ_WAIT_LIMIT_NS": 20000000}, out=out)
    return out


def batches():
    rng = np.random.default_rng(51)
    q = rng.choice([5, 12, 40, 70, 130], 260)
    yield "short segments", q.tolist(), (q + rng.integers(0, 300, 260)).tolist()
    yield "one long chunk", [300], [5000]
    yield "few rows over long contexts", [12, 9, 16], [9000, 7000, 300]
    q = rng.choice([9, 33, 150], 40)
    yield "mixed", q.tolist(), (q + rng.integers(0, 2500, 40)).tolist()


@pytest.mark.parametrize("what,q,lens", list(batches()),
                         ids=lambda x: x if isinstance(x, str) else "")
def test_waits_that_give_up(giving_up, monkeypatch, what, q, lens):
    c = Case(q, lens, hq=4, hkv=1, seed=len(q)).upload()
    ref = c.ref()
    # (what no thread block has written must not be joined)
    ws = kvq.chunk_attention_workspace().fill_(0x7E)
    regular = kvq.LIB_PATH, kvq.lib()
    monkeypatch.setattr(kvq, "LIB_PATH", giving_up)
    monkeypatch.setattr(kvq, "_lib", None)
    c.call(workspace=ws)
    torch.cuda.synchronize()
    assert int(c.err.item()) == kvq.KVQ_DEVERR_TIMEOUT
    got = c.out.double().cpu().numpy()
    left = (got == 77.0).all(-1)               # per row and head
    assert left.any()
    if len(q) > 100:
        assert not left.all()
    c.check(np.where(left[..., None], ref[0], got), ref, what=what)
    monkeypatch.setattr(kvq, "LIB_PATH", regular[0])
    monkeypatch.setattr(kvq, "_lib", regular[1])
    c.err.zero_()
    c.call(workspace=ws)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    c.check(c.out.double().cpu().numpy(), ref, what=what)
