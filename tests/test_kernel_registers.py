"""What the compiler says of the decode attention's kernel (host only): tokens
of short chunks run it in instantiations of their own, which pay for nothing
that trees of drafts and block lists need.  With the masks and the lists in
them they spilled 16 to 44 bytes more than the decode step's and took up to
4 % longer."""
import os
import re

import pytest

from paged_quantized_kv_gb300 import build as kbuild

DECODE, CHUNK, MARKED = 0, 1, 2


@pytest.fixture(scope="module")
def spills():
    """{(heads, fp16, page form, kind of rows): bytes of spill stores}"""
    logs = [os.path.join(kbuild.BUILD, s + ".ptxas") for s in kbuild.SOURCES]
    kbuild.build(force=not all(map(os.path.exists, logs)))
    out, name = {}, None
    for log in logs:
        for line in open(log):
            entry = re.search(r"Compiling entry function '(\S+)'", line)
            if entry:
                name = re.search(r"paged_attention_mma_kernel"
                                 r"ILi(\d+)ELb([01])ELi(\d+)ELi(\d)E",
                                 entry.group(1))
            bytes_ = re.search(r"(\d+) bytes spill stores", line)
            if bytes_ and name:
                out[tuple(map(int, name.groups()))] = int(bytes_.group(1))
    return out


def test_every_kind_of_rows_is_there(spills):
    assert {k[3] for k in spills} == {DECODE, CHUNK, MARKED}
    for kind in (DECODE, CHUNK, MARKED):
        assert len([k for k in spills if k[3] == kind]) == 2 * 2 * 11


def test_chunks_spill_no_more_than_the_decode_step(spills):
    more = {k: (v, spills[(*k[:3], DECODE)]) for k, v in spills.items()
            if k[3] == CHUNK and v > spills[(*k[:3], DECODE)] + 8}
    assert not more
