"""The barriers of the chunk attention's tile kernel in a model (no GPU),
with the ring sizes that the kernel's source has."""
import os
import re

import pytest

from paged_quantized_kv_gb300 import build as kbuild
from tests.chunk_protocol import random_run

with open(os.path.join(kbuild.CSRC, "chunk_attention.cu")) as f:
    SOURCE = f.read()


def ring(name, default):
    """A ring's size in the kernel; a kernel without the constant has
    `default`."""
    found = re.search(rf"constexpr int {name} = (\d+);", SOURCE)
    return int(found.group(1)) if found else default


def faults(kinds, empties, announcements, runs, own_first=True):
    """The kinds of fault (all for None) that random runs find."""
    out = {}
    for seed in range(runs):
        for x in random_run(seed, empties, announcements, own_first):
            if kinds is None or x[0] in kinds:
                out.setdefault(x[:2], (seed, x))
    return out


def test_announced_segments_are_not_missed():
    """Slot 1's softmax warps may still be in the last segment's epilogue
    when the one behind the next is announced."""
    found = faults(("missed", "stuck"), ring("kEmpties", 2),
                   ring("kAnnounced", 1), 1500)
    assert not {k: v for k, v in found.items()
                if k[0] == "missed" and "segment" in k[1]}


def test_the_model_finds_a_single_announcement_barrier():
    found = faults(("missed",), 4, 1, 60)
    assert ("missed", "segment[0]") in found


def test_tiles_are_not_filled_under_their_products():
    """A filler that skips a phase of a tile ring's barrier must not take an
    older one for its own."""
    found = faults(("early", "K under its product", "V under its product",
                    "V at its product"), ring("kEmpties", 2),
                   ring("kAnnounced", 1), 1500)
    assert not {k: v for k, v in found.items() if "o_done" not in str(k[1])}


def test_the_model_finds_a_tile_filled_too_early():
    found = faults(("early", "V under its product"), 2, 2, 60)
    assert any(k[1].startswith("v_empty") for k in found)
    assert any(k[0] == "V under its product" for k in found)


def test_no_fault_of_any_kind():
    """Both slots' results are joined once each slot has waited for its own
    last product; nothing is early, missed, stuck or overwritten."""
    own_first = "kODone + own" in SOURCE
    assert faults(None, ring("kEmpties", 2), ring("kAnnounced", 1), 3000,
                  own_first) == {}


def test_the_model_finds_a_wait_for_the_other_slot():
    found = faults(("early",), 4, 2, 60, own_first=False)
    assert found and all("o_done" in k[1] for k in found)
